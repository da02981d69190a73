"""Thin ctypes binding over libmq.so (C ABI in include/mq.h).

Argument marshalling only: torch tensors in, device pointers and the current
torch stream out; every step of the computation runs in the HIP kernels.
Loading fails loudly when the library has not been built -- there is no host
fallback.  Call ``build()`` (or ``python -m block_quantized_matmul_mq_amd.build``)
first.
"""

import ctypes
import functools
import os

Q4_0 = 2
Q4_1 = 3
Q5_0 = 6
Q5_1 = 7
Q8_0 = 8
Q4_K = 12
Q5_K = 13
Q6_K = 14
REPACKED = 0x100   # OR-ed into Q8_0 / Q6_K / Q4_K: weights in the layout mq_repack writes
ROW_TILED = 0x200  # OR-ed into Q4_K: its row-tiled layout (long-row GEMV), from repack(.., Q4_K | ROW_TILED, ..)

# Activations of gemv_ep / gemm_ep / moe_ffn and router scores of moe_route (include/mq.h)
ACT_NONE, ACT_SILU, ACT_GELU_TANH, ACT_GELU_ERF, ACT_RELU = range(5)
SCORE_SOFTMAX, SCORE_SIGMOID = range(2)

MQ_OK = 0
ERRORS = {
    -1: "MQ_ERR_ARG", -2: "MQ_ERR_SHAPE", -3: "MQ_ERR_TYPE", -4: "MQ_ERR_SIZE",
    -5: "MQ_ERR_ALIGN", -6: "MQ_ERR_DEVICE", -7: "MQ_ERR_LAUNCH", -8: "MQ_ERR_NOINIT",
}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmq.so")

# Every symbol include/mq.h declares, with its ctypes signature.
_SIGNATURES = {
    "mq_init": (ctypes.c_int, [ctypes.c_int]),
    "mq_weight_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64]),
    "mq_act_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "mq_act_scale_offset": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "mq_act_sum_offset": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "mq_act_f6_offset": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "mq_quantize_act": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_void_p]),
    "mq_gemv": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "mq_gemm_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "mq_gemm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                               ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                               ctypes.c_size_t, ctypes.c_void_p]),
    "mq_gemv_ep": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                  ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p]),
    "mq_gemm_ep": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                  ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "mq_gemm_ep_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "mq_moe_route_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "mq_moe_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                    ctypes.c_void_p]),
    "mq_moe_scratch_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "mq_moe_ffn": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int,
                                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                  ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "mq_debug_lds_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int64]),
    "mq_gemm_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "mq_debug_gemm_blockdots": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                               ctypes.c_int64, ctypes.c_void_p]),
    "mq_debug_refuse_launches": (ctypes.c_int, [ctypes.c_int]),
    "mq_repack_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64]),
    "mq_repack": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_size_t,
                                 ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "mq_device_lds_bytes": (ctypes.c_int, []),
    "mq_last_error": (ctypes.c_char_p, []),
    "mq_last_kernel": (ctypes.c_char_p, []),
    "mq_version": (ctypes.c_char_p, []),
}


class MQError(RuntimeError):
    def __init__(self, code, message):
        super().__init__(f"{ERRORS.get(code, code)}: {message}")
        self.code = code


_lib = None


def load():
    """Load libmq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m block_quantized_matmul_mq_amd.build`")
        # torch first: its bundled HIP runtime then also serves libmq (libmq's dependency
        # on libamdhip64.so.7 resolves to the copy already loaded).  Loaded the other way
        # round, the process would hold two HIP runtimes, and the second one to open the
        # device finds none.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def last_error():
    return load().mq_last_error().decode()


def last_kernel():
    return load().mq_last_kernel().decode()


def _check(code):
    if code != MQ_OK:
        raise MQError(code, last_error())


def _nbytes(t):
    return t.numel() * t.element_size()


def _refuse(code, fn, msg):
    raise MQError(code, f"{fn}: {msg}")


def _contiguous(t, fn, name):
    if not t.is_contiguous():
        _refuse(-1, fn, f"{name} must be contiguous")


def _weights(W, qtype, N, K, fn):
    """W must hold exactly the payload of an N x K matrix of qtype (the exact-length gate)."""
    need = weight_bytes(qtype, N, K)
    if need == 0:
        _refuse(-3, fn, f"type {qtype} with N={N} K={K} has no payload size (type or K invalid)")
    _contiguous(W, fn, "W")
    if _nbytes(W) != need:
        _refuse(-4, fn, f"W holds {_nbytes(W)} bytes, an {N} x {K} type-{qtype} payload is exactly {need}")


def _f32(t, numel, fn, name):
    import torch
    if t.dtype is torch.float32 and t.numel() == numel and t.is_contiguous():
        return
    if t.dtype != torch.float32:
        _refuse(-1, fn, f"{name} must be float32, not {t.dtype}")
    _contiguous(t, fn, name)
    if t.numel() != numel:
        _refuse(-4, fn, f"{name} has {t.numel()} elements, {numel} expected")


def _buffer(t, min_bytes, fn, name):
    _contiguous(t, fn, name)
    if _nbytes(t) < min_bytes:
        _refuse(-4, fn, f"{name} holds {_nbytes(t)} bytes, {min_bytes} required")


def _same_device(fn, *tensors):
    d = tensors[0].get_device()      # (-1 on the CPU; no device objects: 0.7 -> 0.3 us per call)
    if d >= 0:
        for t in tensors:
            if t.get_device() != d:
                break
        else:
            return
    devs = {(t.device.type, t.device.index) for t in tensors}
    if len(devs) != 1 or next(iter(devs))[0] != "cuda":
        _refuse(-6, fn, f"every tensor must be on one GPU device, got {sorted(map(str, devs))}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(fn, tensor, stream, *args):
    """fn(*args, stream) on the device of the (checked) tensors, on `stream` or that device's current one."""
    import torch
    # (device and stream without torch's device and stream objects: 3.0 -> 0.3 us per call)
    device = tensor.get_device()
    if device == torch._C._cuda_getDevice():
        code = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream)
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream)
    if code != MQ_OK:
        _check(code)


_GEMM_COUNTER_BYTES, _ROUTE_COUNTER_BYTES = 1024, 256 * 1024    # of the workspaces (include/mq.h)


def _new(stream, like, shape, dtype, zero=0):
    """A tensor on `like`'s device, its first `zero` elements zero, in order on the call's stream: memory that
    the allocator takes back may otherwise be reused, or be cleared, while the call runs."""
    if stream is not None and like.is_cuda:
        import torch
        handle = stream if isinstance(stream, int) else stream.value or 0
        # (0 is the default stream's handle; an ExternalStream of 0 would be a new stream, ordered with nothing)
        on = torch.cuda.ExternalStream(handle, device=like.device) if handle else torch.cuda.default_stream(like.device)
        with torch.cuda.stream(on):
            return _new(None, like, shape, dtype, zero)
    t = like.new_empty(shape, dtype=dtype)
    if zero:
        t[:zero].zero_()
    return t


def init(device=0):
    _check(load().mq_init(device))


# (the sizes are functions of the numbers alone)
@functools.lru_cache(maxsize=4096)
def weight_bytes(qtype, N, K):
    return load().mq_weight_bytes(qtype, N, K)


def repack_bytes(qtype, N, K):
    return load().mq_repack_bytes(qtype, N, K)


def repack(W, qtype, N, K, Wr=None, stream=None):
    """The repacked layout of a GGUF payload W (uint8 CUDA tensor); use with qtype | REPACKED
    (or, for qtype = Q4_K | ROW_TILED, the row-tiled layout; use with Q4_K | ROW_TILED)."""
    import torch
    _weights(W, qtype & ~ROW_TILED, N, K, "repack")
    need = repack_bytes(qtype, N, K)
    if Wr is None:
        Wr = _new(stream, W, need, torch.uint8)
    else:
        _buffer(Wr, need, "repack", "Wr")
    _same_device("repack", W, Wr)
    _call(load().mq_repack, W, stream, W.data_ptr(), qtype, N, K, _nbytes(W), Wr.data_ptr(), _nbytes(Wr))
    return Wr


@functools.lru_cache(maxsize=4096)
def act_bytes(M, K):
    return load().mq_act_bytes(M, K)


def act_layout(M, K):
    """(total bytes, scale offset, sum offset) of the quantized activation plane."""
    lib = load()
    return lib.mq_act_bytes(M, K), lib.mq_act_scale_offset(M, K), lib.mq_act_sum_offset(M, K)


def act_f6(Xq, M, K):
    """View (uint8 [ceil(K/64), 128 * Mp]) of the plane's fp6 section, Mp = M rounded up to 128:
    one slab per 64-value step (layout in include/mq.h)."""
    off = load().mq_act_f6_offset(M, K)
    T = (K + 63) // 64
    Mp = -(-M // 128) * 128
    return Xq[off:off + T * 128 * Mp].view(T, 128 * Mp)


@functools.lru_cache(maxsize=4096)
def gemm_scratch_bytes(qtype, M, N, K):
    return load().mq_gemm_scratch_bytes(qtype, M, N, K)


def quantize_act(X, Xq=None, stream=None):
    """X: f32 [M, K] CUDA tensor -> Xq: uint8 plane of act_bytes(M, K) bytes (made on the call's stream)."""
    import torch
    if X.dim() != 2:
        _refuse(-1, "quantize_act", f"X must be 2-D [M, K], not {tuple(X.shape)}")
    M, K = X.shape
    _f32(X, M * K, "quantize_act", "X")
    need = act_bytes(M, K)
    if need == 0:
        _refuse(-2, "quantize_act", f"K={K} is not a positive multiple of 32")
    if Xq is None:
        Xq = _new(stream, X, need, torch.uint8)
    else:
        _buffer(Xq, need, "quantize_act", "Xq")
    _same_device("quantize_act", X, Xq)
    _call(load().mq_quantize_act, X, stream, X.data_ptr(), Xq.data_ptr(), M, K)
    return Xq


def split_act(Xq, M, K):
    """Views (codes int8 [M, K], scales f32 [M, K/32], sums int32 [M, K/32]) into a plane."""
    import torch
    _, so, uo = act_layout(M, K)
    nb = K // 32
    codes = Xq[:M * K].view(torch.int8).view(M, K)
    scales = Xq[so:so + 4 * M * nb].view(torch.float32).view(M, nb)
    sums = Xq[uo:uo + 4 * M * nb].view(torch.int32).view(M, nb)
    return codes, scales, sums


def gemv(W, qtype, x, N, K, y=None, stream=None):
    """y[N] = deq(W) @ x for a uint8 GGUF payload W and f32 x[K] (CUDA tensors)."""
    import torch
    _weights(W, qtype, N, K, "gemv")
    _f32(x, K, "gemv", "x")
    if y is None:
        y = _new(stream, x, N, torch.float32)
    else:
        _f32(y, N, "gemv", "y")
    _same_device("gemv", W, x, y)
    _call(load().mq_gemv, x, stream, W.data_ptr(), qtype, x.data_ptr(), y.data_ptr(), N, K)
    return y


def _act_plane(Xq, M, K, fn):
    need = act_bytes(M, K)
    if need == 0:
        _refuse(-2, fn, f"M={M} K={K}: K is not a positive multiple of 32")
    _buffer(Xq, need, fn, "Xq")


def gemm(W, qtype, Xq, M, N, K, Y=None, scratch=None, stream=None):
    """Y[M, N] from a quantized activation plane Xq and weights W (CUDA tensors)."""
    import torch
    _weights(W, qtype, N, K, "gemm")
    _act_plane(Xq, M, K, "gemm")
    if Y is None:
        Y = _new(stream, Xq, (M, N), torch.float32)
    else:
        _f32(Y, M * N, "gemm", "Y")
    need = gemm_scratch_bytes(qtype, M, N, K)
    if scratch is None and need:
        scratch = _new(stream, Xq, need, torch.uint8, zero=_GEMM_COUNTER_BYTES)
    tensors = [W, Xq, Y]
    if scratch is not None:
        _buffer(scratch, need, "gemm", "scratch")
        tensors.append(scratch)
    _same_device("gemm", *tensors)
    _call(load().mq_gemm, Xq, stream, W.data_ptr(), qtype, Xq.data_ptr(), Y.data_ptr(), M, N, K, _ptr(scratch),
          0 if scratch is None else _nbytes(scratch))
    return Y


def gemm_noalloc(W, qtype, Xq, M, N, K, Y, stream=None):
    """mq_gemm_noalloc: the product into a caller-provided Y, with the library's own
    per-device scratch (the call allocates nothing; overlapping calls on one device race)."""
    _weights(W, qtype, N, K, "gemm_noalloc")
    _act_plane(Xq, M, K, "gemm_noalloc")
    _f32(Y, M * N, "gemm_noalloc", "Y")
    _same_device("gemm_noalloc", W, Xq, Y)
    _call(load().mq_gemm_noalloc, Xq, stream, W.data_ptr(), qtype, Xq.data_ptr(), Y.data_ptr(), M, N, K)
    return Y


def gemm_blockdots(W, qtype, Xq, M, N, K, D=None, stream=None):
    """Exact int32 block dots [M, N, G] of the MMQ kernel (G = K/32, or K/16 for Q6_K)."""
    import torch
    _weights(W, qtype, N, K, "gemm_blockdots")
    _act_plane(Xq, M, K, "gemm_blockdots")
    G = K // 16 if (qtype & ~REPACKED) == Q6_K else K // 32
    if D is None:
        D = _new(stream, Xq, (M, N, G), torch.int32)
    else:
        if D.dtype != torch.int32:
            _refuse(-1, "gemm_blockdots", f"D must be int32, not {D.dtype}")
        _contiguous(D, "gemm_blockdots", "D")
        if D.numel() != M * N * G:
            _refuse(-4, "gemm_blockdots", f"D has {D.numel()} elements, {M * N * G} expected")
    _same_device("gemm_blockdots", W, Xq, D)
    _call(load().mq_debug_gemm_blockdots, Xq, stream, W.data_ptr(), qtype, Xq.data_ptr(), D.data_ptr(), M, N, K)
    return D


def _terms(fn, M, N, bias, mul, residual):
    """The epilogue's tensors that are given, checked."""
    given = []
    for t, numel, name in ((bias, N, "bias"), (mul, M * N, "mul"), (residual, M * N, "residual")):
        if t is not None:
            _f32(t, numel, fn, name)
            given.append(t)
    return given


def gemv_ep(W, qtype, x, N, K, bias=None, act=ACT_NONE, mul=None, residual=None, y=None, stream=None):
    """y[N] = act(deq(W) @ x + bias) * mul + residual, one launch (bias, mul, residual: f32 [N] or None;
    y may be mul or residual)."""
    import torch
    _weights(W, qtype, N, K, "gemv_ep")
    _f32(x, K, "gemv_ep", "x")
    given = _terms("gemv_ep", 1, N, bias, mul, residual)
    if y is None:
        y = _new(stream, x, N, torch.float32)
    else:
        _f32(y, N, "gemv_ep", "y")
    _same_device("gemv_ep", W, x, y, *given)
    _call(load().mq_gemv_ep, x, stream, W.data_ptr(), qtype, x.data_ptr(), y.data_ptr(), N, K, _ptr(bias), act, _ptr(mul),
          _ptr(residual))
    return y


@functools.lru_cache(maxsize=4096)
def gemm_ep_scratch_bytes(qtype, M, N, K):
    return load().mq_gemm_ep_scratch_bytes(qtype, M, N, K)


def gemm_ep(W, qtype, Xq, M, N, K, bias=None, act=ACT_NONE, mul=None, residual=None, Y=None, scratch=None,
            stream=None):
    """Y[M, N] = act(product + bias) * mul + residual, the product of gemm (bias: f32 [N]; mul, residual:
    f32 [M, N]; each may be None; Y may be mul or residual).  scratch: gemm_scratch_bytes, or
    gemm_ep_scratch_bytes for its own work split; its first KiB zero before its first use."""
    import torch
    _weights(W, qtype, N, K, "gemm_ep")
    _act_plane(Xq, M, K, "gemm_ep")
    given = _terms("gemm_ep", M, N, bias, mul, residual)
    if Y is None:
        Y = _new(stream, Xq, (M, N), torch.float32)
    else:
        _f32(Y, M * N, "gemm_ep", "Y")
    if scratch is None:
        need = gemm_ep_scratch_bytes(qtype, M, N, K)
        if need:
            scratch = _new(stream, Xq, need, torch.uint8, zero=_GEMM_COUNTER_BYTES)
            given.append(scratch)
    else:
        _buffer(scratch, gemm_scratch_bytes(qtype, M, N, K), "gemm_ep", "scratch")
        given.append(scratch)
    _same_device("gemm_ep", W, Xq, Y, *given)
    _call(load().mq_gemm_ep, Xq, stream, W.data_ptr(), qtype, Xq.data_ptr(), Y.data_ptr(), M, N, K, _ptr(bias), act,
          _ptr(mul), _ptr(residual), _ptr(scratch), 0 if scratch is None else _nbytes(scratch))
    return Y


def _i32(t, numel, fn, name):
    import torch
    if t.dtype != torch.int32:
        _refuse(-1, fn, f"{name} must be int32, not {t.dtype}")
    _contiguous(t, fn, name)
    if t.numel() != numel:
        _refuse(-4, fn, f"{name} has {t.numel()} elements, {numel} expected")


def _rows(X, fn):
    if X.dim() != 2:
        _refuse(-1, fn, f"X must be 2-D [M, K], not {tuple(X.shape)}")
    return X.shape


@functools.lru_cache(maxsize=4096)
def moe_route_scratch_bytes(M, K, E):
    return load().mq_moe_route_scratch_bytes(M, K, E)


def moe_route(X, Wr, topk, bias=None, score=SCORE_SOFTMAX, norm=True, scale=1.0, ids=None, wts=None, scratch=None,
              stream=None):
    """(ids int32 [M, topk], wts f32 [M, topk]) of tokens X (f32 [M, K]) by router weights Wr (f32 [E, K]);
    bias: f32 [E], added to the scores for the choice only.  scratch: moe_route_scratch_bytes(M, K, E) bytes,
    zero before its first use, and for calls of moe_route only."""
    import torch
    M, K = _rows(X, "moe_route")
    E = Wr.shape[0]
    _f32(X, M * K, "moe_route", "X")
    _f32(Wr, E * K, "moe_route", "Wr")
    need = moe_route_scratch_bytes(M, K, E)
    if scratch is None:
        scratch = _new(stream, X, max(need, 16), torch.uint8, zero=_ROUTE_COUNTER_BYTES)
    else:
        _buffer(scratch, need, "moe_route", "scratch")
    tensors = [X, Wr, scratch]
    if bias is not None:
        _f32(bias, E, "moe_route", "bias")
        tensors.append(bias)
    if ids is None:
        ids = _new(stream, X, (M, topk), torch.int32)
    else:
        _i32(ids, M * topk, "moe_route", "ids")
    if wts is None:
        wts = _new(stream, X, (M, topk), torch.float32)
    else:
        _f32(wts, M * topk, "moe_route", "wts")
    _same_device("moe_route", ids, wts, *tensors)
    _call(load().mq_moe_route, X, stream, X.data_ptr(), Wr.data_ptr(), _ptr(bias), ids.data_ptr(), wts.data_ptr(), M, K, E,
          topk, score, int(norm), scale, scratch.data_ptr(), _nbytes(scratch))
    return ids, wts


@functools.lru_cache(maxsize=4096)
def moe_scratch_bytes(M, topk, F, K):
    return load().mq_moe_scratch_bytes(M, topk, F, K)


def moe_ffn(Wg, Wu, gu_type, Wd, d_type, X, ids, wts, E, F, act=ACT_SILU, residual=None, Y=None, scratch=None,
            stream=None):
    """Y[M, K] = residual + sum_j wts[:, j] * down_e(act(gate_e(X)) * up_e(X)), e = ids[:, j]: a
    mixture-of-experts feed-forward layer for a few tokens.  Wg, Wu: E matrices of F x K weights, Wd: E of
    K x F (uint8 payloads); ids int32 and wts f32 [M, topk].  scratch: moe_scratch_bytes(M, topk, F, K) bytes."""
    import torch
    M, K = _rows(X, "moe_ffn")
    _f32(X, M * K, "moe_ffn", "X")
    _weights(Wg, gu_type, E * F, K, "moe_ffn")
    _weights(Wu, gu_type, E * F, K, "moe_ffn")
    _weights(Wd, d_type, E * K, F, "moe_ffn")
    if ids.dim() != 2 or ids.shape[0] != M:
        _refuse(-1, "moe_ffn", f"ids must be [M, topk] with M={M}, not {tuple(ids.shape)}")
    topk = ids.shape[1]
    _i32(ids, M * topk, "moe_ffn", "ids")
    _f32(wts, M * topk, "moe_ffn", "wts")
    tensors = [Wg, Wu, Wd, X, ids, wts]
    if residual is not None:
        _f32(residual, M * K, "moe_ffn", "residual")
        tensors.append(residual)
    if Y is None:
        Y = _new(stream, X, (M, K), torch.float32)
    else:
        _f32(Y, M * K, "moe_ffn", "Y")
    need = moe_scratch_bytes(M, topk, F, K)
    if scratch is None:
        scratch = _new(stream, X, max(need, 16), torch.uint8)
    else:
        _buffer(scratch, need, "moe_ffn", "scratch")
    _same_device("moe_ffn", Y, scratch, *tensors)
    _call(load().mq_moe_ffn, X, stream, Wg.data_ptr(), Wu.data_ptr(), gu_type, Wd.data_ptr(), d_type, X.data_ptr(),
          ids.data_ptr(), wts.data_ptr(), _ptr(residual), Y.data_ptr(), M, topk, E, F, K, act, scratch.data_ptr(),
          _nbytes(scratch))
    return Y
