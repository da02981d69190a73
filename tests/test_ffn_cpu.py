"""CPU checks of the feed-forward operators: sizes and refusals before any HIP call, and the oracle
functions that the GPU tests compare with, pinned by values worked by hand and by brute force."""

import math

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth

FAKE = 0x10000
BIG = 1 << 40


def gemv_ep(W=FAKE, t=mq.Q4_K, x=FAKE, y=FAKE, N=8, K=256, bias=None, act=0, mul=None, res=None):
    return mq.load().mq_gemv_ep(W, t, x, y, N, K, bias, act, mul, res, None)


def gemm_ep(W=FAKE, t=mq.Q4_K, Xq=FAKE, Y=FAKE, M=4, N=8, K=256, bias=None, act=0, mul=None, res=None, s=None, sb=0):
    return mq.load().mq_gemm_ep(W, t, Xq, Y, M, N, K, bias, act, mul, res, s, sb, None)


def route(X=FAKE, Wr=FAKE, bias=None, ids=FAKE, wts=FAKE, M=4, K=64, E=8, k=2, score=0, norm=1, s=FAKE, sb=BIG):
    return mq.load().mq_moe_route(X, Wr, bias, ids, wts, M, K, E, k, score, norm, 1.0, s, sb, None)


def ffn(Wg=FAKE, Wu=FAKE, gu=mq.Q4_K, Wd=FAKE, d=mq.Q6_K, X=FAKE, ids=FAKE, wts=FAKE, res=None, Y=FAKE, M=4, k=2, E=8,
        F=256, K=512, act=1, s=FAKE, sb=BIG):
    return mq.load().mq_moe_ffn(Wg, Wu, gu, Wd, d, X, ids, wts, res, Y, M, k, E, F, K, act, s, sb, None)


def test_epilogue_refusals():
    assert gemv_ep(W=None) == -1 and gemv_ep(y=None) == -1
    assert gemv_ep(act=5) == -1 and gemv_ep(act=-1) == -1
    assert "activation" in mq.last_error() and "mq_gemv_ep" in mq.last_error()
    assert gemv_ep(K=128) == -2 and gemv_ep(t=10) == -3 and gemv_ep(t=mq.Q4_K | mq.REPACKED) == -3
    assert gemv_ep(bias=FAKE + 2) == -5 and gemv_ep(mul=FAKE + 1) == -5 and gemv_ep(res=FAKE + 3) == -5
    assert gemv_ep(x=FAKE + 8) == -5
    assert gemm_ep(Y=None) == -1 and gemm_ep(act=7) == -1 and gemm_ep(M=0) == -1
    assert gemm_ep(K=96) == -2 and gemm_ep(t=11) == -3 and gemm_ep(t=mq.Q4_K | mq.ROW_TILED, K=17 * 256, M=40) == -3
    assert gemm_ep(mul=FAKE + 2) == -5 and gemm_ep(Xq=FAKE + 16) == -5
    need = mq.gemm_scratch_bytes(mq.Q8_0, 512, 512, 3584)
    big = dict(t=mq.Q8_0, M=512, N=512, K=3584)
    assert need > 0 and gemm_ep(**big) == -4 and gemm_ep(s=FAKE, sb=need - 1, **big) == -4
    assert gemm_ep(s=FAKE + 4, sb=need, **big) == -5


def test_epilogue_scratch():
    """gemm_ep's own work split: 1 KiB of counters and a partial tile for each of at most 512 workgroups."""
    def tiles(count, splits, rows):
        return 1024 + count * splits * rows * 128 * 4

    size = mq.gemm_ep_scratch_bytes
    assert size(mq.Q6_K, 333, 5120, 13824) == tiles(120, 4, 128)
    assert size(mq.Q8_0, 512, 8192, 8192) == tiles(256, 2, 128)
    assert size(mq.Q5_1, 64, 8192, 8192) == tiles(128, 4, 32)
    assert size(mq.Q8_0, 512, 3584, 3584) == 0 == mq.gemm_scratch_bytes(mq.Q8_0, 512, 3584, 3584)
    for t in (mq.Q4_0, mq.Q4_1, mq.Q5_0, mq.Q5_1, mq.Q8_0, mq.Q4_K, mq.Q5_K, mq.Q6_K):
        block = 256 if t in (mq.Q4_K, mq.Q5_K, mq.Q6_K) else 32
        for M in (1, 8, 9, 31, 33, 100, 129, 333, 512, 1000, 4096):
            for N in (1, 130, 1000, 4096, 8200, 18944):
                for K in (block, 7 * 256, 3584, 8192, 32768):
                    plain, own = mq.gemm_scratch_bytes(t, M, N, K), size(t, M, N, K)
                    assert plain <= own <= 1024 + (32 << 20) or own == plain, (t, M, N, K)
    plane = mq.Q4_K | mq.REPACKED
    assert size(plane, 512, 18944, 3584) == mq.gemm_scratch_bytes(plane, 512, 18944, 3584)
    assert size(mq.Q4_K, 0, 10, 256) == size(mq.Q4_K, 40, 10, 100) == size(99, 40, 10, 256) == 0
    assert size(mq.Q4_K | mq.ROW_TILED, 40, 10, 256) == 0


def test_route_sizes_and_refusals():
    size = mq.moe_route_scratch_bytes
    assert size(0, 64, 8) == size(4, 48, 8) == size(4, 64, 0) == size(4, 64, 513) == size(1, 1 << 16, 8) == 0
    # counters (256 KiB), then f64 partial logits of 16-token tiles
    assert size(1, 64, 8) == (1 << 18) + 16 * 8 * 8
    assert size(4096, 4096, 128) == (1 << 18) + 4096 * 128 * 8
    for name in ("X", "Wr", "ids", "wts", "s"):
        assert route(**{name: None}) == -1, name
    assert route(M=0) == -1 and route(k=0) == -1 and route(E=-3) == -1 and route(score=2) == -1
    assert route(K=40) == -2 and route(K=1 << 16) == -2 and route(E=513, k=2) == -2 and route(M=(1 << 20) + 1) == -2
    assert route(k=9) == -2 and route(E=100, k=65) == -2
    assert route(sb=size(4, 64, 8) - 1) == -4
    assert route(X=FAKE + 4) == -5 and route(Wr=FAKE + 8) == -5 and route(bias=FAKE + 1) == -5 and route(ids=FAKE + 2) == -5
    assert "mq_moe_route" in mq.last_error()


def test_moe_sizes_and_refusals():
    size = mq.moe_scratch_bytes
    assert size(0, 2, 256, 512) == size(1, 0, 256, 512) == size(2049, 2, 256, 512) == size(1, 1, 1 << 16, 512) == 0
    assert size(1, 8, 256, 512) == 8 * 256 * 4                        # h of every pair
    assert size(16, 8, 256, 512) == 2 * 128 * 256 * 4 + 128 * 512 * 4     # its two factors, and the weighted rows
    for name in ("Wg", "Wu", "Wd", "X", "ids", "wts", "Y", "s"):
        assert ffn(**{name: None}) == -1, name
    assert ffn(M=0) == -1 and ffn(k=-1) == -1 and ffn(E=0) == -1 and ffn(act=9) == -1 and ffn(F=0) == -1
    assert ffn(gu=10) == -3 and ffn(d=99) == -3
    assert ffn(gu=mq.Q4_K | mq.REPACKED) == -3 and ffn(d=mq.Q4_K | mq.ROW_TILED) == -3 and ffn(d=mq.Q4_0 | mq.REPACKED) == -3
    assert ffn(K=320) == -2                       # gate / up rows: a multiple of 256
    assert ffn(F=288) == -2                       # down rows
    assert ffn(F=256, K=(1 << 15) + 256) == -2 and ffn(F=(1 << 15) + 256) == -2
    assert ffn(E=513) == -2 and ffn(M=2048, k=3) == -2 and ffn(M=1 << 62, k=8) == -2
    assert ffn(sb=size(4, 2, 256, 512) - 1) == -4
    for name in ("Wg", "Wu", "Wd", "X", "Y", "s", "res"):
        assert ffn(**{name: FAKE + 8}) == -5, name
    assert ffn(ids=FAKE + 2) == -5 and "mq_moe_ffn" in mq.last_error()


def test_calls_without_init_are_refused():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    for call in (gemv_ep, gemm_ep, route, ffn):
        assert call() in (-6, -8), call.__name__


def test_binding_refuses_bad_tensors():
    import torch
    W = torch.zeros(8 * 144, dtype=torch.uint8)
    x, n = torch.zeros(256), torch.zeros(8)

    def code(fn, *a, **k):
        with pytest.raises(mq.MQError) as e:
            fn(*a, **k)
        return e.value.code

    assert code(mq.gemv_ep, W, mq.Q4_K, x, 8, 256, bias=torch.zeros(7)) == -4
    assert code(mq.gemv_ep, W, mq.Q4_K, x, 8, 256, mul=n.double()) == -1
    assert code(mq.gemv_ep, W, mq.Q4_K, x, 8, 256, residual=torch.zeros(16)[::2]) == -1
    assert code(mq.gemv_ep, W[:-1], mq.Q4_K, x, 8, 256) == -4
    assert code(mq.gemv_ep, W, mq.Q4_K, x, 8, 256) == -6            # CPU tensors
    X = torch.zeros((2, 64))
    Wr = torch.zeros((8, 64))
    assert code(mq.moe_route, X[0], Wr, 2) == -1
    assert code(mq.moe_route, X, Wr[:, :32].contiguous(), 2) == -4
    assert code(mq.moe_route, X, Wr, 2, bias=torch.zeros(9)) == -4
    assert code(mq.moe_route, X, Wr, 2, ids=torch.zeros((2, 2), dtype=torch.int64)) == -1
    assert code(mq.moe_route, X, Wr, 2, scratch=torch.zeros(16, dtype=torch.uint8)) == -4
    assert code(mq.moe_route, X, Wr, 2) == -6
    X = torch.zeros((2, 256))
    P = torch.zeros(2 * 256 * 144, dtype=torch.uint8)
    ids, wts = torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2))
    args = (P, P, mq.Q4_K, P, mq.Q4_K)
    assert code(mq.moe_ffn, *args, X, ids, wts, 3, 256) == -4                      # three experts' payload
    assert code(mq.moe_ffn, *args, X, ids.long(), wts, 2, 256) == -1
    assert code(mq.moe_ffn, *args, X, ids[:1], wts, 2, 256) == -1
    assert code(mq.moe_ffn, *args, X, ids, wts[:, :1].contiguous(), 2, 256) == -4
    assert code(mq.moe_ffn, *args, X, ids, wts, 2, 256, scratch=torch.zeros(16, dtype=torch.uint8)) == -4
    assert code(mq.moe_ffn, *args, X, ids, wts, 2, 256) == -6


# ------------------------------------------------------------------ the oracle

def test_oracle_activations_by_hand():
    v = np.array([-30.0, -2.0, 0.0, 1.0, 3.0])
    assert np.array_equal(oracle.activation(v, 0), v)
    assert np.array_equal(oracle.activation(v, 4), [0, 0, 0, 1, 3])
    for x in v:
        assert math.isclose(oracle.activation(x, 1), x / (1 + math.exp(-x)), rel_tol=1e-12, abs_tol=1e-14)
        assert math.isclose(oracle.activation(x, 3), 0.5 * x * math.erfc(-x / math.sqrt(2)), rel_tol=1e-12, abs_tol=0)
        t = math.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
        assert math.isclose(oracle.activation(x, 2), 0.5 * x * (1 + t), rel_tol=1e-12, abs_tol=1e-14)
    # the slope bound that the expert layer's error bound uses
    g = np.linspace(-20, 20, 400001)
    for act in range(5):
        assert np.abs(np.diff(oracle.activation(g, act)) / np.diff(g)).max() <= 1.13


def test_oracle_epilogue_order():
    acc, b, m, r = np.array([[2.0, -3.0]]), np.array([1.0, 1.0]), np.array([[2.0, 5.0]]), np.array([[10.0, 20.0]])
    assert np.array_equal(oracle.epilogue(acc, b, 4, m, r), [[16.0, 20.0]])      # relu before mul before residual
    assert np.array_equal(oracle.epilogue(acc, None, 0, None, None), acc)


def test_oracle_route_by_hand():
    X = np.array([[1.0, 0.0], [0.0, 2.0]])
    Wr = np.array([[0.0, 1.0], [math.log(3), 1.0], [math.log(3), 0.0], [0.0, 0.0]])
    ids, w = oracle.moe_route(X, Wr, 2)
    assert np.array_equal(ids, [[1, 2], [0, 1]])                      # ties: the lower index
    assert np.allclose(w, [[0.5, 0.5], [0.5, 0.5]])
    ids, w = oracle.moe_route(X[:1], Wr, 4, norm=False, scale=8.0)
    assert np.allclose(w, [[3, 3, 1, 1]])                             # 8 p, p = 3/8, 3/8, 1/8, 1/8
    ids, w = oracle.moe_route(X[:1], Wr, 1, bias=[9, 0, 0, 0], score=1, norm=False)
    assert ids[0, 0] == 0 and np.allclose(w, 0.5)                     # the bias chooses, the weight is sigmoid(0)


def test_oracle_moe_by_brute_force():
    E, F, K, M, k = 3, 32, 64, 2, 2
    rng = np.random.default_rng(3)
    g, u = (synth.random_blocks(mq.Q8_0, E * F, K, rng) for _ in range(2))
    d = synth.random_blocks(mq.Q4_0, E * K, F, rng)
    X = rng.standard_normal((M, K)).astype(np.float32)
    ids, wts = np.array([[2, 0], [-1, 2]]), np.array([[0.25, 2.0], [5.0, -1.0]])
    Y, bound = oracle.moe_ffn(g, u, mq.Q8_0, d, mq.Q4_0, X, ids, wts, E, F, residual=X)
    Wg, Wu = (oracle.decode(w, mq.Q8_0, E * F, K).reshape(E, F, K) for w in (g, u))
    Wd = oracle.decode(d, mq.Q4_0, E * K, F).reshape(E, K, F)
    for m in range(M):
        for n in range(K):
            y = float(X[m, n])
            for j in range(k):
                e = ids[m, j]
                if e < 0:
                    continue
                for f in range(F):
                    a = sum(Wg[e, f, i] * float(X[m, i]) for i in range(K))
                    b = sum(Wu[e, f, i] * float(X[m, i]) for i in range(K))
                    y += wts[m, j] * Wd[e, n, f] * (a / (1 + math.exp(-a)) if a > -700 else 0.0) * b
            assert math.isclose(Y[m, n], y, rel_tol=1e-9, abs_tol=1e-12 * np.abs(Y).max())
    assert np.all(bound > 0) and np.all(bound < 1e-3 * np.abs(Y).max())


@pytest.mark.parametrize("qtype", [mq.Q4_K, mq.Q5_K, mq.Q4_1, mq.Q5_1, mq.Q8_0])
def test_oracle_magnitude_bounds_the_weights(qtype):
    raw = synth.random_blocks(qtype, 5, 256, np.random.default_rng(4))
    w, mag = oracle.decode(raw, qtype, 5, 256), oracle.magnitude(raw, qtype, 5, 256)
    assert np.all(mag >= np.abs(w) * (1 - 1e-12)) and np.all(mag <= 1e3 * np.abs(w).max())
