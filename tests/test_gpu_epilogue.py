"""GPU parity of mq_gemv_ep and mq_gemm_ep, on every kernel that they run.

* Without terms they give the bits of mq_gemv / mq_gemm, but for what is formed more precisely here: mq_gemv's
  offset and min terms (from the staged activations) and mq_gemm's min terms on the int8 kernels (to f32
  precision); there the f64 product within the bound of f32 sums.
* With terms the result is the oracle's epilogue of that accumulator, within the roundings of the
  epilogue's own f32 steps.
"""

import itertools

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import ALL_TYPES, BLOCK, NAMES, device, say, to_dev, weights

pytestmark = pytest.mark.gpu

ACTS = {mq.ACT_NONE: "none", mq.ACT_SILU: "silu", mq.ACT_GELU_TANH: "gelu_tanh", mq.ACT_GELU_ERF: "gelu_erf",
        mq.ACT_RELU: "relu"}
HALF = 2.0 ** -24    # half a step of f32


def terms_bound(acc, bias, act, mul, residual):
    """How far f32 steps may be from oracle.epilogue: the bias addition (half a step of the sum,
    times an activation's slope, at most 1.13), the activation (exp, erfc and the division within 16 half steps;
    an exponent's relative error multiplies by the argument, at most |v| + v^2 + |v|^3 / 10 with four half steps),
    one half step for each later operation."""
    v = acc.astype(np.float64) + (0 if bias is None else bias.astype(np.float64))
    a = oracle.activation(v, act)
    w = np.abs(v)
    err = 1.13 * HALF * w * (bias is not None) + (act != 0) * (16 + 4 * (w + w ** 2 + 0.1 * w ** 3)) * HALF * np.abs(a)
    err = err + 2.0 ** -126 * (act != 0)      # (an exp that overflows: the quotient rounds to 0)
    if mul is not None:
        err = err * np.abs(mul) + 2 * HALF * np.abs(a * mul)
        a = a * mul
    if residual is not None:
        err = err * 1.01 + HALF * np.abs(a + residual.astype(np.float64))
    return err


def combos():
    for act, (b, m, r) in itertools.product(ACTS, itertools.product((False, True), repeat=3)):
        if act == mq.ACT_SILU or (b, m, r) in ((True, False, False), (True, True, True)) or (act == 0 and (b or m or r)):
            yield act, b, m, r


def check_terms(call, acc, M, N, what):
    """call(**terms) against the epilogue of acc (f32 [M, N])."""
    import torch
    dev = device()
    rng = np.random.default_rng(N + M)
    bias = (rng.standard_normal(N) * 2).astype(np.float32)
    mul = rng.standard_normal((M, N)).astype(np.float32)
    res = rng.standard_normal((M, N)).astype(np.float32)
    for act, b, m, r in combos():
        t = dict(bias=bias if b else None, mul=mul if m else None, residual=res if r else None)
        y = call(act=act, **{k: None if v is None else to_dev(v, dev) for k, v in t.items()})
        torch.cuda.synchronize()
        y = y.cpu().numpy().reshape(M, N)
        ref = oracle.epilogue(acc, t["bias"], act, t["mul"], t["residual"])
        err = np.abs(y - ref)
        bound = terms_bound(acc, t["bias"], act, t["mul"], t["residual"])
        assert np.all(err <= bound), f"{what} {ACTS[act]} {b, m, r}: {float((err / np.maximum(bound, 1e-300)).max())}"


GEMV = [  # (type, N, K, kernel)
    *[(t, 37, 3 * BLOCK[t], "gemv<" + NAMES[t] + ">") for t in ALL_TYPES],
    (mq.Q4_K, 8224, 3584, "gemv_mfma<q4_K>"),
    (mq.Q4_K, 16400, 3584, "gemv_mfma<q4_K>"),
    (mq.Q4_K, 2100, 17 * 256, "gemv_mfma_long<q4_K>"),
    (mq.Q4_K | mq.ROW_TILED, 700, 17 * 256, "gemv_mfma_long<q4_K row-tiled>"),
    (mq.Q6_K, 8200, 3584, "gemv_mfma<q6_K>"),
    (mq.Q8_0, 8201, 3584, "gemv_mfma<q8_0>"),
    (mq.Q4_0, 8201, 3584, "gemv_mfma<q4_0>"),
    (mq.Q5_0, 8201, 3584, "gemv_mfma<q5_0>"),
    (mq.Q8_0 | mq.REPACKED, 45, 96, "gemv<q8_0 repacked>"),
    (mq.Q6_K | mq.REPACKED, 45, 512, "gemv<q6_K repacked>"),
]


def laid_out(raw, qtype, N, K, dev):
    W = to_dev(raw.reshape(-1), dev)
    if qtype & mq.ROW_TILED:
        return mq.repack(W, qtype, N, K)
    return mq.repack(W, qtype & ~mq.REPACKED, N, K) if qtype & mq.REPACKED else W


@pytest.mark.parametrize("qtype,N,K,kernel", GEMV, ids=[f"{g[3]}-{g[1]}x{g[2]}" for g in GEMV])
def test_gemv(qtype, N, K, kernel):
    import torch
    dev = device()
    say(f"gemv_ep {kernel} N={N} K={K}")
    raw = weights(qtype & 0xFF, N, K, "quantized", 700)
    W = laid_out(raw, qtype, N, K, dev)
    X = synth.activations(1, K, config_index=14, tensor_index=7)
    x = to_dev(X[0], dev)
    acc = mq.gemv(W, qtype, x, N, K)
    assert mq.last_kernel() == kernel, mq.last_kernel()
    y = mq.gemv_ep(W, qtype, x, N, K)
    assert mq.last_kernel() == kernel
    torch.cuda.synchronize()
    acc, plain = y.cpu().numpy(), acc.cpu().numpy()
    base = qtype & 0xFF
    if base == mq.Q8_0:
        assert np.array_equal(acc, plain)
    else:
        # x staged within 2^-21 of its block's largest (half a unit, the largest at least 2^20 units), met by the
        # weight; K / 32 block terms and their offset or min terms, summed in f32 (any order), each product rounded
        w = oracle.decode(raw, base, N, K)
        top = np.abs(X.reshape(-1, 32)).max(1).astype(np.float64).repeat(32)
        bound = 2.0 ** -21 * (np.abs(w) @ top) + (K / 32 + 24) * HALF * (oracle.magnitude(raw, base, N, K) @ np.abs(X[0]))
        ref = w @ X[0].astype(np.float64)
        err = np.abs(acc - ref)
        rel = [float(np.linalg.norm(v - ref) / np.linalg.norm(ref)) for v in (acc, plain)]
        say(f"  worst error / bound {float((err / bound).max()):.3f}, relative {rel[0]:.2e} (mq_gemv {rel[1]:.2e})")
        assert np.all(err <= bound)
    check_terms(lambda **t: mq.gemv_ep(W, qtype, x, N, K, **t), acc[None], 1, N, kernel)


GEMM = [  # (type, M, N, K, kernel)
    *[(t, 5, 37, 2 * BLOCK[t], "gemv_q8<" + NAMES[t] + ">") for t in ALL_TYPES],
    (mq.Q6_K, 3, 8200, 3584, "gemv_q8_mfma<q6_K>"),
    (mq.Q6_K, 8, 8200, 3584, "gemv_q8_mfma<q6_K>"),
    *[(t, 40, 300, 2 * BLOCK[t], "mmq<" + NAMES[t] + ">") for t in ALL_TYPES if t != mq.Q4_K],
    *[(t, 33, 130, 4096, "mmq<" + NAMES[t] + ">") for t in (mq.Q8_0, mq.Q6_K, mq.Q5_K, mq.Q4_1)],   # K cut
    (mq.Q4_K, 40, 100, 8192, "mmq<q4_K>"),                                                          # K cut
    (mq.Q4_K, 300, 14000, 256, "mmq<q4_K>"),                                                        # 128-row tiles
    (mq.Q5_1, 300, 14000, 64, "mmq<q5_1>"),
    (mq.Q4_K, 40, 300, 512, "mmq_kw<q4_K>"),
    (mq.Q4_K, 70, 513, 3584, "mmq_kw<q4_K>"),
    (mq.Q4_K | mq.REPACKED, 40, 300, 512, "mmq_f6<q4_K plane>"),
    (mq.Q4_K | mq.REPACKED, 200, 300, 8192, "mmq_f6<q4_K plane>"),
    (mq.Q8_0 | mq.REPACKED, 40, 300, 96, "mmq<q8_0 repacked>"),
]


@pytest.mark.parametrize("qtype,M,N,K,kernel", GEMM, ids=[f"{g[4]}-{g[1]}x{g[2]}x{g[3]}" for g in GEMM])
def test_gemm(qtype, M, N, K, kernel):
    import torch
    dev = device()
    say(f"gemm_ep {kernel} M={M} N={N} K={K}")
    base = qtype & 0xFF
    raw = weights(base, N, K, "quantized", 710)
    W = laid_out(raw, qtype, N, K, dev)
    X = synth.activations(M, K, config_index=14, tensor_index=8)
    Xq = mq.quantize_act(to_dev(X, dev))
    scratch = torch.zeros(max(16, mq.gemm_scratch_bytes(qtype, M, N, K)), dtype=torch.uint8, device=dev)
    plain = mq.gemm(W, qtype, Xq, M, N, K, scratch=scratch)
    assert mq.last_kernel() == kernel, mq.last_kernel()
    Y = mq.gemm_ep(W, qtype, Xq, M, N, K, scratch=scratch)
    assert mq.last_kernel() == kernel
    torch.cuda.synchronize()
    acc = Y.cpu().numpy()
    if base in (mq.Q4_K, mq.Q5_K, mq.Q4_1, mq.Q5_1) and kernel.startswith(("mmq<", "mmq_kw")):
        # K / 32 block terms and their min terms, summed in f32 (any order), each product rounded
        q, d, _ = oracle.quantize_act(X)
        ref = oracle.mmq(raw, base, q, d, N, K)
        xh = np.abs(q.reshape(M, -1, 32) * d[..., None].astype(np.float64)).reshape(M, K)
        bound = (K / 32 + 24) * HALF * (xh @ oracle.magnitude(raw, base, N, K).T)
        err = np.abs(acc - ref)
        say(f"  worst error / bound {float((err / bound).max()):.3f}, relative {np.linalg.norm(acc - ref) / np.linalg.norm(ref):.2e}")
        assert np.all(err <= bound)
    else:
        assert np.array_equal(acc, plain.cpu().numpy())
    check_terms(lambda **t: mq.gemm_ep(W, qtype, Xq, M, N, K, scratch=scratch, **t), acc, M, N, kernel)


FILLED = [  # (type, M, N, K, tile rows of the split)
    (mq.Q6_K, 333, 5120, 4096, 128), (mq.Q8_0, 200, 4100, 8192, 128), (mq.Q4_0, 384, 2047, 8192, 128),
    (mq.Q4_K, 333, 8190, 8192, 128), (mq.Q5_1, 64, 8192, 4096, 32), (mq.Q5_0, 128, 4096, 4096 + 32, 32),
    (mq.Q4_1, 30, 16001, 4096, 32), (mq.Q5_K, 9, 8000, 8192, 32), (mq.Q8_0 | mq.REPACKED, 137, 3155, 8192, 32),
]


@pytest.mark.parametrize("qtype,M,N,K,rows", FILLED, ids=[f"{NAMES[f[0] & 0xFF]}-{f[1]}x{f[2]}x{f[3]}" for f in FILLED])
def test_gemm_with_its_own_split(qtype, M, N, K, rows):
    """With gemm_ep_scratch_bytes of scratch the tiles are cut into other K ranges: the f64 product within
    the bound of f32 sums, the same bits from call to call (with other bytes in the partial tiles), and the
    counters left at zero; with less, mq_gemm's split."""
    import torch
    dev = device()
    base = qtype & 0xFF
    say(f"gemm_ep own split {NAMES[base]} M={M} N={N} K={K}")
    need, plain = mq.gemm_ep_scratch_bytes(qtype, M, N, K), mq.gemm_scratch_bytes(qtype, M, N, K)
    tile_bytes = -(-M // rows) * -(-N // 128) * rows * 128 * 4
    assert need > plain and (need - 1024) % tile_bytes == 0 and (need - 1024) // tile_bytes >= 2
    raw = weights(base, N, K, "quantized", 720)
    W = laid_out(raw, qtype, N, K, dev)
    X = synth.activations(M, K, config_index=14, tensor_index=9)
    Xq = mq.quantize_act(to_dev(X, dev))
    own = torch.zeros(need, dtype=torch.uint8, device=dev)
    Y = mq.gemm_ep(W, qtype, Xq, M, N, K, scratch=own)
    assert mq.last_kernel().startswith("mmq<")
    own[1024:] = 255     # (f32 NaN)
    again = mq.gemm_ep(W, qtype, Xq, M, N, K, scratch=own)
    alone = mq.gemm_ep(W, qtype, Xq, M, N, K)
    less = mq.gemm_ep(W, qtype, Xq, M, N, K, scratch=torch.zeros(max(plain, 16), dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert int(own[:1024].sum()) == 0
    assert torch.equal(Y, again) and torch.equal(Y, alone)
    # K / 32 block terms and their min terms, summed in f32 (any order), each product rounded; some columns
    cols = np.unique(np.concatenate([np.arange(min(N, 40)), np.arange(max(0, N - 140), N), np.arange(0, N, 97)]))
    q, d, _ = oracle.quantize_act(X)
    part = np.ascontiguousarray(raw.reshape(N, -1)[cols])
    ref = oracle.mmq(part, base, q, d, len(cols), K)
    xh = np.abs(q.reshape(M, -1, 32) * d[..., None].astype(np.float64)).reshape(M, K)
    bound = (K / 32 + 24) * HALF * (xh @ oracle.magnitude(part, base, len(cols), K).T)
    for y in (Y, less):
        acc = y.cpu().numpy()[:, cols]
        err = np.abs(acc - ref)
        say(f"  worst error / bound {float((err / bound).max()):.3f}, relative {np.linalg.norm(acc - ref) / np.linalg.norm(ref):.2e}")
        assert np.all(err <= bound)
    acc = Y.cpu().numpy()
    rng = np.random.default_rng(M)
    mul, res = rng.standard_normal((M, N)).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    y = mq.gemm_ep(W, qtype, Xq, M, N, K, act=mq.ACT_SILU, mul=to_dev(mul, dev), residual=to_dev(res, dev), scratch=own)
    err = np.abs(y.cpu().numpy() - oracle.epilogue(acc, None, mq.ACT_SILU, mul, res))
    assert np.all(err <= terms_bound(acc, None, mq.ACT_SILU, mul, res))


def test_the_output_may_be_a_term():
    import torch
    dev = device()
    N, K, M = 300, 512, 40
    W = to_dev(weights(mq.Q4_K, N, K, "quantized", 720).reshape(-1), dev)
    X = to_dev(synth.activations(M, K, config_index=14, tensor_index=9), dev)
    Xq = mq.quantize_act(X)
    rng = np.random.default_rng(1)
    res, mul = rng.standard_normal((M, N)).astype(np.float32), rng.standard_normal((M, N)).astype(np.float32)
    want = mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, act=mq.ACT_SILU, mul=to_dev(mul, dev), residual=to_dev(res, dev))
    for term in ("mul", "residual"):
        t = dict(mul=to_dev(mul, dev), residual=to_dev(res, dev))
        mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, act=mq.ACT_SILU, Y=t[term], **t)
        assert torch.equal(t[term], want)
    same = to_dev(res, dev)      # one buffer as multiplier, residual and output
    mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, mul=same, residual=same, Y=same)
    other = mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, mul=to_dev(res, dev), residual=to_dev(res, dev))
    assert torch.equal(same, other)
    y = to_dev(res[0], dev)
    want = mq.gemv_ep(W, mq.Q4_K, X[0].contiguous(), N, K, residual=to_dev(res[0], dev))
    mq.gemv_ep(W, mq.Q4_K, X[0].contiguous(), N, K, residual=y, y=y)
    assert torch.equal(y, want)
    # K cut over workgroups: only the piece that finishes reads the terms
    N, K = 100, 8192
    W = to_dev(weights(mq.Q4_K, N, K, "quantized", 721).reshape(-1), dev)
    Xq = mq.quantize_act(to_dev(synth.activations(M, K, config_index=14, tensor_index=10), dev))
    res = to_dev(rng.standard_normal((M, N)).astype(np.float32), dev)
    want = mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, residual=res.clone())
    mq.gemm_ep(W, mq.Q4_K, Xq, M, N, K, residual=res, Y=res)
    assert torch.equal(res, want)


def test_non_finite_terms_stay_where_they_are():
    import torch
    dev = device()
    N, K = 64, 256
    W = to_dev(weights(mq.Q4_K, N, K, "quantized", 730).reshape(-1), dev)
    x = to_dev(synth.activations(1, K, config_index=14, tensor_index=11)[0], dev)
    clean = mq.gemv_ep(W, mq.Q4_K, x, N, K, act=mq.ACT_SILU)
    bias = torch.zeros(N, device=dev)
    bias[3], bias[4], bias[5] = float("nan"), float("inf"), 1e30
    y = mq.gemv_ep(W, mq.Q4_K, x, N, K, bias=bias, act=mq.ACT_SILU)
    assert torch.isnan(y[3]) and y[4] == float("inf") and y[5] == 1e30
    keep = [i for i in range(N) if i not in (3, 4, 5)]
    assert torch.equal(y[keep], clean[keep])
    bias[:] = -1e30          # silu and gelu of a very negative number are 0, not NaN
    for act in (mq.ACT_SILU, mq.ACT_GELU_TANH, mq.ACT_GELU_ERF, mq.ACT_RELU):
        assert torch.all(mq.gemv_ep(W, mq.Q4_K, x, N, K, bias=bias, act=act) == 0), ACTS[act]
