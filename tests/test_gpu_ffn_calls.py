"""How the feed-forward calls (mq_gemv_ep, mq_gemm_ep, mq_moe_route, mq_moe_ffn) run rather than what they
compute: refused launches, a raw stream without buffers of the caller's, two calls at once, weights
beyond 4 GiB, many tokens, and the workspaces they leave behind."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import device, say, to_dev, weights

pytestmark = pytest.mark.gpu

E, K, F, TOPK = 8, 512, 256, 3


def experts(qtype, rows, cols, count, seed):
    rng = np.random.default_rng(8100 + seed)
    return synth.random_blocks(qtype, count * rows, cols, rng, exp_lo=-12, exp_hi=-8).reshape(count, -1)


class Calls:
    """Each of the four calls with inputs of its own on the device; run(name, **kw) gives its outputs."""

    def __init__(self, M=5, seed=0):
        dev = device()
        rng = np.random.default_rng(900 + seed)
        normal = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32), dev)   # noqa: E731
        self.M = M
        self.X, self.x = normal(M, K), normal(K)
        self.N = 300
        self.W = to_dev(weights(mq.Q4_K, self.N, K, "random", 70 + seed).reshape(-1), dev)
        self.Xg = normal(40, K)
        self.Xq = mq.quantize_act(self.Xg)
        self.mul, self.mulg = normal(self.N), normal(40, self.N)
        self.Wr = normal(E, K) * 0.1
        self.g, self.u = (to_dev(experts(mq.Q4_K, F, K, E, seed + i).reshape(-1), dev) for i in (0, 1))
        self.d = to_dev(experts(mq.Q6_K, K, F, E, seed + 2).reshape(-1), dev)
        self.ids = to_dev(rng.integers(0, E, (M, TOPK)).astype(np.int32), dev)
        self.wts = to_dev(rng.random((M, TOPK)).astype(np.float32), dev)

    def gemv_ep(self, **kw):
        return (mq.gemv_ep(self.W, mq.Q4_K, self.x, self.N, K, act=mq.ACT_SILU, mul=self.mul, **kw),)

    def gemm_ep(self, **kw):
        return (mq.gemm_ep(self.W, mq.Q4_K, self.Xq, 40, self.N, K, act=mq.ACT_SILU, mul=self.mulg, **kw),)

    def moe_route(self, **kw):
        return mq.moe_route(self.X, self.Wr, TOPK, **kw)

    def moe_ffn(self, **kw):
        return (mq.moe_ffn(self.g, self.u, mq.Q4_K, self.d, mq.Q6_K, self.X, self.ids, self.wts, E, F, **kw),)


NAMES = ("gemv_ep", "gemm_ep", "moe_route", "moe_ffn")


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_launch_is_reported_and_leaves_nothing_behind(name):
    import torch
    lib = mq.load()
    c = Calls()
    say(f"refused launch: {name}")
    before = getattr(c, name)()
    assert lib.mq_debug_refuse_launches(1) == 0
    with pytest.raises(mq.MQError) as e:
        getattr(c, name)()
    assert e.value.code == -7, e.value
    msg = mq.last_error()
    assert f"mq_{name}: launch of" in msg and "refused" in msg and "hipErrorLaunchFailure" in msg, msg
    after = getattr(c, name)()
    torch.cuda.synchronize()
    for a, b in zip(before, after):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_handle_without_buffers(name):
    """The binding's own outputs and workspaces belong to the stream it is given: the current stream is
    kept busy meanwhile, and its freed memory holds other values."""
    import torch
    c = Calls(seed=1)
    ref = getattr(c, name)()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=c.X.device)
    for turn in range(3):
        say(f"{name} on a stream handle, call {turn}")
        for _ in range(4):
            busy = (busy @ busy).clamp_(-1, 1)
        junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=c.X.device) for _ in range(4)]
        del junk
        out = getattr(c, name)(stream=s.cuda_stream)
        s.synchronize()
        for a, b in zip(ref, out):
            assert torch.equal(a, b), turn
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("M", [1, 5])
def test_two_calls_at_once(name, M):
    import torch
    a, b = Calls(M, seed=2), Calls(M, seed=3)
    refs = getattr(a, name)(), getattr(b, name)()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    say(f"{name} M={M} on two streams")
    outs = [[], []]
    for _ in range(20):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                outs[i].append(getattr(c, name)())
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            for x, y in zip(refs[i], o):
                assert torch.equal(x, y)


@pytest.mark.parametrize("M,k", [(1, 4), (3, 4), (40, 2)])
def test_experts_beyond_4_gib(M, k):
    """512 experts whose payloads pass 2^32 bytes: the first and the last ones give the bits of a layer that
    holds only those."""
    import torch
    big, width, hidden = 512, 4096, 2048
    some = (0, 1, big - 2, big - 1)
    dev = device()
    rows = ((hidden, width), (hidden, width), (width, hidden))
    small = [experts(mq.Q8_0, r, c, len(some), 40 + i) for i, (r, c) in enumerate(rows)]
    assert big * small[0].shape[1] > 2 ** 32
    W = []
    for s in small:
        w = torch.zeros((big, s.shape[1]), dtype=torch.uint8, device=dev)
        for i, e in enumerate(some):
            w[e].copy_(to_dev(s[i], dev))
        W.append(w.reshape(-1))
    rng = np.random.default_rng(5)
    X = to_dev(rng.standard_normal((M, width)).astype(np.float32), dev)
    pick = np.stack([rng.permutation(len(some))[:k] for _ in range(M)]).astype(np.int32)
    wts = to_dev(rng.random((M, k)).astype(np.float32), dev)
    say(f"moe M={M} with {big} experts, {W[0].numel() / 2 ** 30:.2f} GiB a matrix")
    Y = mq.moe_ffn(W[0], W[1], mq.Q8_0, W[2], mq.Q8_0, X, to_dev(np.array(some, np.int32)[pick], dev), wts, big, hidden)
    D = [to_dev(s.reshape(-1), dev) for s in small]
    Ys = mq.moe_ffn(D[0], D[1], mq.Q8_0, D[2], mq.Q8_0, X, to_dev(pick, dev), wts, len(some), hidden)
    torch.cuda.synchronize()
    assert torch.equal(Y, Ys) and bool(torch.isfinite(Y).all()) and float(Y.abs().max()) > 0


def test_router_of_many_tokens():
    import torch
    dev = device()
    M, width, count, k = 20011, 64, 24, 6
    rng = np.random.default_rng(6)
    X = rng.standard_normal((M, width)).astype(np.float32)
    Wr = rng.standard_normal((count, width)).astype(np.float32)
    scratch = torch.zeros(mq.moe_route_scratch_bytes(M, width, count), dtype=torch.uint8, device=dev)
    say(f"route M={M}")
    ids, wts = mq.moe_route(to_dev(X, dev), to_dev(Wr, dev), k, scratch=scratch)
    torch.cuda.synchronize()
    ref_ids, ref = oracle.moe_route(X, Wr, k)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    # one rounding to f32, doubled for the f64 steps
    assert np.all(np.abs(wts.cpu().numpy() - ref) <= 2.0 ** -23 * np.abs(ref))
    assert int(scratch[:256 * 1024].sum()) == 0     # the counters, as every call leaves them


@pytest.mark.parametrize("M", [1, 5])
def test_nothing_is_written_past_the_outputs(M):
    """Guard values around the outputs and behind the workspaces stay."""
    import torch
    c = Calls(M, seed=4)
    dev = c.X.device

    def guarded(numel, dtype):
        buf = torch.full((numel + 128,), 77, dtype=dtype, device=dev)
        return buf, buf[64:64 + numel]

    say(f"guards M={M}")
    bufs = []

    def take(numel, dtype, zero=False):
        buf, view = guarded(numel, dtype)
        if zero:
            view.zero_()
        bufs.append((buf, numel))
        return view

    f32, i32, u8 = torch.float32, torch.int32, torch.uint8
    c.gemv_ep(y=take(c.N, f32))
    c.gemm_ep(Y=take(40 * c.N, f32).view(40, c.N))
    c.moe_route(ids=take(M * TOPK, i32).view(M, TOPK), wts=take(M * TOPK, f32).view(M, TOPK),
                scratch=take(mq.moe_route_scratch_bytes(M, K, E), u8, zero=True))
    c.moe_ffn(Y=take(M * K, f32).view(M, K), scratch=take(mq.moe_scratch_bytes(M, TOPK, F, K), u8))
    torch.cuda.synchronize()
    for buf, numel in bufs:
        assert bool((buf[:64] == 77).all()) and bool((buf[64 + numel:] == 77).all())
