"""mq_moe_ffn where its launches take other forms than the usual four tokens per slot: rows so long that fewer
tokens' activations fit in LDS (three at 40 groups of 256 values of Q8_0, one at 128), few (token, choice) pairs, the
longest rows of the one-token kernels; and one token with every special input that the batch is tested with."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq

from gpu_cases import NAMES, say, to_dev
from test_gpu_moe import Layer, inputs

pytestmark = pytest.mark.gpu

ACTS = [mq.ACT_NONE, mq.ACT_SILU, mq.ACT_GELU_TANH, mq.ACT_GELU_ERF, mq.ACT_RELU]
# (type, F, K): a long K is the up kernel's row, a long F the down kernel's
LONG = [(mq.Q8_0, 64, 10240), (mq.Q8_0, 64, 16384), (mq.Q8_0, 32, 32768), (mq.Q8_0, 10240, 64), (mq.Q8_0, 16384, 32),
        (mq.Q8_0, 32768, 32), (mq.Q6_K, 256, 10240), (mq.Q6_K, 10240, 256), (mq.Q6_K, 256, 32768),
        (mq.Q4_K, 256, 12288), (mq.Q4_K, 32768, 256), (mq.Q5_1, 32, 32768 - 32), (mq.Q5_1, 32768 - 32, 32)]
LAYERS = {}


def layer(qtype, F, K, E=3):
    """(kept for the module's tests of the same layer, one at a time)"""
    key = (qtype, F, K, E)
    if key not in LAYERS:
        LAYERS.clear()
        LAYERS[key] = Layer(qtype, qtype, E, F, K, seed=200 + qtype)
    return LAYERS[key]


def against_oracle(lay, Y, X, ids, wts, tokens, what, residual=None):
    ref, bound = oracle.moe_ffn(lay.raw[0], lay.raw[1], lay.gu, lay.raw[2], lay.down, X[tokens], ids[tokens], wts[tokens], lay.E,
                                lay.F, residual=None if residual is None else residual[tokens])
    err = np.abs(Y[tokens] - ref)
    say(f"  {what}: worst error / bound {float((err / np.where(bound > 0, bound, 1.0)).max()):.3f}")
    assert np.all(err <= bound), what


@pytest.mark.parametrize("M,k", [(1, 2), (6, 3), (40, 3)])
@pytest.mark.parametrize("qtype,F,K", LONG, ids=[f"{NAMES[t]}-F{f}-K{k}" for t, f, k in LONG])
def test_rows_longer_than_four_tokens_of_lds(qtype, F, K, M, k):
    """Against the oracle, and the bits of the same tokens in other slots: pairs of tokens by themselves."""
    say(f"moe long rows {NAMES[qtype]} M={M} k={k} F={F} K={K}")
    lay = layer(qtype, F, K)
    X, ids, wts = inputs(M, k, 3, K, 30 + M, distinct=False)
    if M > 1:
        ids[0] = [1, -1, 1]
        ids[M - 1, 0] = 3
    res = np.random.default_rng(6).standard_normal((M, K)).astype(np.float32)
    Y = lay.run(X, ids, wts, residual=res)
    assert mq.last_kernel() == ("moe_one" if M == 1 else "moe_many")
    tokens = np.unique([0, M - 1] if F * K < 1 << 22 else [M - 1])    # (decoding is slow on the CPU)
    against_oracle(lay, Y, X, ids, wts, tokens, "against the oracle", res)
    for m in range(0, M - 1, 1 if M < 10 else 13):
        part = slice(m, m + 2)
        assert np.array_equal(lay.run(X[part], ids[part], wts[part], residual=res[part]), Y[part]), m


@pytest.mark.parametrize("M,k", [(2, 1), (3, 1), (1, 65), (5, 1), (1, 66), (1, 67)])
def test_few_pairs(M, k):
    """Slots of two, three or four pairs, all of one expert and of several."""
    E, F, K = 5, 256, 512
    lay = Layer(mq.Q4_K, mq.Q8_0, E, F, K, seed=210)
    for same in (False, True):
        X, ids, wts = inputs(M, k, E, K, 40 + M + k, distinct=False)
        if same:
            ids[:] = 4
        lay.check(X, ids, wts, what=f"same expert: {same}")


# ------------------------------------------------------------------ one token

E1, F1, K1 = 6, 512, 768


@pytest.fixture(scope="module")
def one():
    return Layer(mq.Q4_K, mq.Q6_K, E1, F1, K1, seed=220)


@pytest.mark.parametrize("act", ACTS)
def test_one_token_activations(one, act):
    X, ids, wts = inputs(1, 4, E1, K1, 50)
    one.check(X, ids, wts, act=act)


@pytest.mark.parametrize("k", [1, 3, 64])
def test_one_token_invalid_ids_add_nothing(one, k):
    X, ids, wts = inputs(1, k, E1, K1, 51, distinct=False)
    res = np.random.default_rng(7).standard_normal((1, K1)).astype(np.float32)
    clean = one.check(X, ids, wts, residual=res)
    if k > 1:
        kept = ids[:, :1].copy(), wts[:, :1].copy()
        ids[0, 1:] = [(-1, E1, -2147483648, 2147483647)[i % 4] for i in range(k - 1)]
        wts[0, 1:] = np.nan            # weights of dropped choices are not read into the sum
        Y = one.check(X, ids, wts, residual=res)
        ref, bound = oracle.moe_ffn(one.raw[0], one.raw[1], one.gu, one.raw[2], one.down, X, *kept, E1, F1, residual=res)
        assert np.all(np.abs(Y - ref) <= bound)
    ids[:] = -1
    wts[:] = np.inf
    assert np.array_equal(one.run(X, ids, wts, residual=res), res)
    assert np.all(one.run(X, ids, wts) == 0)
    assert np.all(np.isfinite(clean))


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("at", [0, 255, 700, K1 - 1])
def test_one_token_non_finite_input(one, value, at):
    X, ids, wts = inputs(1, 3, E1, K1, 52)
    res = np.zeros((1, K1), np.float32)
    X[0, at] = value
    assert np.all(np.isnan(one.run(X, ids, wts)))
    assert np.all(np.isnan(one.run(X, ids, wts, residual=res)))
    ids[:] = -1                        # no expert reads it
    assert np.all(one.run(X, ids, wts, residual=res) == 0)


def test_one_token_overflow_in_the_hidden_layer(one):
    """act(g) * u past f32's range: NaN or infinite as the documentation has it, not a finite number."""
    X, ids, wts = inputs(1, 2, E1, K1, 53)
    assert np.all(np.isnan(one.run(X * np.float32(1e25), ids, wts, act=mq.ACT_NONE)))


def test_one_token_non_finite_weight(one):
    X, ids, wts = inputs(1, 2, E1, K1, 54)
    wts[0, 1] = np.nan
    assert np.all(np.isnan(one.run(X, ids, wts)))


def test_one_token_zero_tiny_and_large_activations(one):
    X, ids, wts = inputs(1, 3, E1, K1, 55)
    assert np.all(one.check(np.zeros_like(X), ids, wts) == 0)
    one.check(X * np.float32(1e-25), ids, wts)
    one.check(X * np.float32(1e4), ids, wts)
    X[0, 7] = 1e6
    X[0, 256:512] = 0
    one.check(X, ids, wts)


def test_one_token_output_may_be_input_or_residual(one):
    import torch
    X, ids, wts = inputs(1, 4, E1, K1, 56)
    res = np.random.default_rng(8).standard_normal((1, K1)).astype(np.float32)
    args = (one.W[0], one.W[1], one.gu, one.W[2], one.down)
    d = one.dev

    def into(x, residual, Y):
        mq.moe_ffn(*args, x, to_dev(ids, d), to_dev(wts, d), E1, F1, residual=residual, Y=Y)
        torch.cuda.synchronize()
        return Y.cpu().numpy()

    buf = to_dev(res, d)
    assert np.array_equal(into(to_dev(X, d), buf, buf), one.run(X, ids, wts, residual=res))
    x = to_dev(X, d)
    assert np.array_equal(into(x, None, x), one.run(X, ids, wts))
    x = to_dev(X, d)
    assert np.array_equal(into(x, x, x), one.run(X, ids, wts, residual=X))
    x, buf = to_dev(X, d), to_dev(res, d)
    assert np.array_equal(into(x, buf, x), one.run(X, ids, wts, residual=res))


def test_one_token_scratch_needs_no_initial_value(one):
    import torch
    X, ids, wts = inputs(1, 5, E1, K1, 57)
    ids[0, 2] = -1
    ref = one.run(X, ids, wts)
    for fill in (0, 255):
        scratch = torch.full((mq.moe_scratch_bytes(1, 5, F1, K1),), fill, dtype=torch.uint8, device=one.dev)
        assert np.array_equal(one.run(X, ids, wts, scratch=scratch), ref)
