"""GPU parity of mq_moe_route against the oracle's f64 router: the ids exactly, the weights to f32
rounding (f64 arithmetic, one rounding at the end: 2^-24 relative, doubled for the f64 steps)."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq

from gpu_cases import device, say, to_dev

pytestmark = pytest.mark.gpu


def run(X, Wr, k, bias=None, **kw):
    import torch
    dev = device()
    say(f"route M={X.shape[0]} K={X.shape[1]} E={Wr.shape[0]} k={k} {kw if 'scratch' not in kw else ''}")
    ids, wts = mq.moe_route(to_dev(X, dev), to_dev(Wr, dev), k, bias=None if bias is None else to_dev(bias, dev), **kw)
    torch.cuda.synchronize()
    assert mq.last_kernel() == "moe_route"
    return ids.cpu().numpy(), wts.cpu().numpy()


def check(X, Wr, k, bias=None, **kw):
    ids, wts = run(X, Wr, k, bias, **kw)
    kw.pop("scratch", None)
    ref_ids, ref = oracle.moe_route(X, Wr, k, bias, **kw)
    assert np.array_equal(ids, ref_ids)
    assert np.all(np.abs(wts - ref) <= 2.0 ** -23 * np.abs(ref) + 1e-45)
    return ids, wts


def inputs(M, K, E, seed):
    rng = np.random.default_rng(seed)
    X = rng.standard_normal((M, K)).astype(np.float32)
    Wr = (rng.standard_normal((E, K)) * 2 / np.sqrt(K)).astype(np.float32)
    return X, Wr, (rng.standard_normal(E) * 0.1).astype(np.float32)


@pytest.mark.parametrize("M,K,E,k", [(1, 32, 1, 1), (1, 2048, 64, 8), (3, 96, 7, 7), (17, 640, 60, 4), (16, 352, 33, 2),
                                     (33, 1024, 128, 8), (100, 256, 160, 6), (70, 512, 257, 10), (5, 256, 512, 64),
                                     (600, 128, 16, 2)])
@pytest.mark.parametrize("score", [mq.SCORE_SOFTMAX, mq.SCORE_SIGMOID], ids=["softmax", "sigmoid"])
def test_shapes(M, K, E, k, score):
    X, Wr, bias = inputs(M, K, E, M + E)
    check(X, Wr, k, score=score, norm=True)
    check(X, Wr, k, bias=bias, score=score, norm=False, scale=2.5)


def test_ties_go_to_the_lowest_index():
    X, Wr, _ = inputs(20, 128, 200, 1)
    Wr[150] = Wr[3]          # equal rows: equal logits
    Wr[67] = Wr[3]
    Wr[131] = Wr[130]
    check(X, Wr, 64)
    ids, _ = check(X, np.zeros_like(Wr), 9)
    assert np.array_equal(ids, np.tile(np.arange(9), (20, 1)))
    X[0] = 0                 # logits of -0 and 0 are equal
    check(X, Wr, 5)


def test_near_ties_in_f32_are_told_apart():
    """Logits that agree to 2^-30: an f32 sum could not order them."""
    rng = np.random.default_rng(2)
    K, E = 1024, 64
    X = rng.standard_normal((8, K)).astype(np.float32)
    base = rng.standard_normal(K).astype(np.float32)
    Wr = np.tile(base, (E, 1))
    Wr[:, 0] = base[0] + (rng.permutation(E) * 2.0 ** -20).astype(np.float32)
    check(X, Wr, 8)


def test_selection_bias_masks_experts():
    X, Wr, bias = inputs(9, 256, 12, 3)
    bias[[0, 5, 11]] = -np.inf
    ids, _ = check(X, Wr, 4, bias=bias, score=mq.SCORE_SIGMOID)
    assert not np.isin(ids, [0, 5, 11]).any()
    bias[:] = -np.inf        # nothing left to choose by: the lowest indices, weights by score
    ids, _ = check(X, Wr, 4, bias=bias, score=mq.SCORE_SIGMOID)
    assert np.array_equal(ids, np.tile(np.arange(4), (9, 1)))
    bias[:] = 0
    bias[7] = np.inf
    ids, _ = check(X, Wr, 4, bias=bias)
    assert np.all(ids[:, 0] == 7)


def test_non_finite_logits_stay_in_their_token():
    X, Wr, _ = inputs(18, 128, 40, 4)
    clean, cw = run(X, Wr, 5)
    X[2, 3] = np.nan
    X[17, 0] = np.inf
    ids, wts = run(X, Wr, 5)
    rest = [i for i in range(18) if i not in (2, 17)]
    assert np.array_equal(ids[rest], clean[rest]) and np.array_equal(wts[rest], cw[rest])
    for m in (2, 17):        # ids stay valid and different
        assert ((ids[m] >= 0) & (ids[m] < 40)).all() and len(set(ids[m])) == 5
    Wr[6] = np.nan           # an expert whose logits are NaN is chosen after every number
    ids, _ = run(X[:2], Wr, 40)
    assert np.all(ids[:, 39] == 6)


def test_large_logits():
    X, Wr, _ = inputs(4, 256, 32, 5)
    check(X * 300, Wr, 4)
    check(X * 300, Wr, 4, norm=False)


def test_scratch_is_reused_over_shapes_and_streams_of_calls():
    import torch
    dev = device()
    shapes = [(1, 2048, 64, 8), (300, 512, 128, 8), (17, 256, 9, 2)]
    need = max(mq.moe_route_scratch_bytes(M, K, E) for M, K, E, _ in shapes)
    scratch = torch.zeros(need, dtype=torch.uint8, device=dev)
    for turn in range(3):
        for M, K, E, k in shapes:
            X, Wr, _ = inputs(M, K, E, 10 * turn + E)
            check(X, Wr, k, scratch=scratch)
    assert int(scratch[:256 * 1024].sum()) == 0


def test_deterministic():
    X, Wr, _ = inputs(40, 4096, 128, 6)
    a = run(X, Wr, 8)
    for _ in range(3):
        b = run(X, Wr, 8)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("E", [40, 130, 512])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("score", [mq.SCORE_SOFTMAX, mq.SCORE_SIGMOID], ids=["softmax", "sigmoid"])
def test_weights_of_non_finite_logits(E, norm, score):
    """An expert whose logit is NaN is in the softmax of every expert: its token's weights are NaN, chosen or not,
    normalized or not; a sigmoid is NaN for that expert alone.  Infinite logits as the formula has them."""
    rng = np.random.default_rng(11)
    M, K = 5, 64
    X = np.abs(rng.standard_normal((M, K))).astype(np.float32)
    Wr = (rng.standard_normal((E, K)) * 0.2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)

    def same(Wr, bias, k):
        ids, wts = run(X, Wr, k, bias, score=score, norm=norm)
        with np.errstate(all="ignore"):
            ref_ids, ref = oracle.moe_route(X, Wr, k, bias, score=score, norm=norm)
        assert np.array_equal(ids, ref_ids)
        assert np.array_equal(np.isnan(wts), np.isnan(ref)), (wts, ref)
        ok = ~np.isnan(ref)
        assert np.all(np.abs(wts[ok] - ref[ok]) <= 2.0 ** -23 * np.abs(ref[ok]) + 1e-45)
        return wts

    for value in (np.nan, np.inf, -np.inf):
        bad = Wr.copy()
        bad[6] = value
        for k in (1, 5, min(E, 64)):
            w = same(bad, None, k)
            if np.isnan(value) and score == mq.SCORE_SOFTMAX:
                assert np.all(np.isnan(w))
        same(bad, bias, 5)
    same(np.full_like(Wr, -np.inf), None, 3)
