"""GPU parity of mq_moe_ffn against the oracle's f64 expert layer, within the oracle's derived
bound (22-bit activations per block, every f32 rounding counted)."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import ALL_TYPES, BLOCK, NAMES, device, say, to_dev

pytestmark = pytest.mark.gpu


def experts(qtype, rows, cols, E, seed):
    """uint8 [E, rows * row bytes] of random blocks (each expert its own)."""
    rng = np.random.default_rng(7000 + seed)
    return synth.random_blocks(qtype, E * rows, cols, rng, exp_lo=-12, exp_hi=-8).reshape(E, -1)


class Layer:
    def __init__(self, gu, down, E, F, K, seed=0):
        self.gu, self.down, self.E, self.F, self.K = gu, down, E, F, K
        self.raw = [experts(gu, F, K, E, seed), experts(gu, F, K, E, seed + 1), experts(down, K, F, E, seed + 2)]
        self.dev = device()
        self.W = [to_dev(r.reshape(-1), self.dev) for r in self.raw]

    def run(self, X, ids, wts, act=mq.ACT_SILU, residual=None, **kw):
        import torch
        d = self.dev
        Y = mq.moe_ffn(self.W[0], self.W[1], self.gu, self.W[2], self.down, to_dev(X, d), to_dev(ids, d), to_dev(wts, d),
                       self.E, self.F, act=act, residual=None if residual is None else to_dev(residual, d), **kw)
        torch.cuda.synchronize()
        return Y.cpu().numpy()

    def check(self, X, ids, wts, act=mq.ACT_SILU, residual=None, what=""):
        M, k = ids.shape
        say(f"moe {NAMES[self.gu]}/{NAMES[self.down]} M={M} k={k} E={self.E} F={self.F} K={self.K} {what}")
        Y = self.run(X, ids, wts, act, residual)
        assert mq.last_kernel() == ("moe_one" if M == 1 and k <= 64 else "moe_many")
        ref, bound = oracle.moe_ffn(self.raw[0], self.raw[1], self.gu, self.raw[2], self.down, X, ids, wts, self.E, self.F,
                                    act, residual)
        err = np.abs(Y - ref)
        worst = float((err / np.where(bound > 0, bound, 1.0)).max())
        rel = float(np.linalg.norm(Y - ref) / max(np.linalg.norm(ref), 1e-300))
        say(f"  worst error / bound {worst:.3f}, relative {rel:.2e}")
        assert np.all(err <= bound), f"{what}: {worst}"
        return Y


def inputs(M, k, E, K, seed, distinct=True):
    rng = np.random.default_rng(seed)
    X = rng.standard_normal((M, K)).astype(np.float32)
    if distinct:
        ids = np.stack([rng.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    else:
        ids = rng.integers(0, E, (M, k)).astype(np.int32)
    wts = (rng.random((M, k)) + 0.1).astype(np.float32)
    return X, ids, wts


@pytest.mark.parametrize("qtype", ALL_TYPES, ids=[NAMES[t] for t in ALL_TYPES])
@pytest.mark.parametrize("M,k", [(1, 2), (3, 3), (7, 2), (20, 2), (33, 1)])
def test_every_type(qtype, M, k):
    b = BLOCK[qtype]
    E, F, K = 5, (256 if b == 256 else 160), (512 if b == 256 else 352)
    X, ids, wts = inputs(M, k, E, K, 11 * M + k)
    res = np.random.default_rng(3).standard_normal((M, K)).astype(np.float32)
    Layer(qtype, qtype, E, F, K, seed=3 * qtype).check(X, ids, wts, residual=res)


@pytest.mark.parametrize("gu,down", [(mq.Q4_K, mq.Q6_K), (mq.Q4_K, mq.Q8_0), (mq.Q8_0, mq.Q4_K), (mq.Q6_K, mq.Q5_0)],
                         ids=["q4_K-q6_K", "q4_K-q8_0", "q8_0-q4_K", "q6_K-q5_0"])
@pytest.mark.parametrize("M", [1, 9])
def test_mixed_types(gu, down, M):
    X, ids, wts = inputs(M, 4, 8, 768, 5)
    Layer(gu, down, 8, 256, 768, seed=50).check(X, ids, wts)


@pytest.mark.parametrize("act", [mq.ACT_NONE, mq.ACT_SILU, mq.ACT_GELU_TANH, mq.ACT_GELU_ERF, mq.ACT_RELU])
def test_activations(act):
    X, ids, wts = inputs(2, 2, 4, 256, 6)
    Layer(mq.Q4_K, mq.Q4_K, 4, 256, 256, seed=60).check(X, ids, wts, act=act)


def test_sizes_of_one_block():
    X, ids, wts = inputs(1, 1, 1, 32, 7)
    Layer(mq.Q8_0, mq.Q4_0, 1, 32, 32, seed=70).check(X, ids, wts)
    X, ids, wts = inputs(40, 1, 1, 32, 8)      # forty tokens of one expert: five chunks of eight
    Layer(mq.Q8_0, mq.Q4_0, 1, 32, 32, seed=71).check(X, ids, wts)


@pytest.mark.parametrize("M,k", [(1, 4), (2, 16), (3, 16), (8, 16), (8, 17), (64, 2)])
def test_long_rows_take_phases(M, k):
    # rows of many 256-value groups: more than fit the staging LDS at once
    E, F, K = 6, 2560, 5120
    X, ids, wts = inputs(M, k, E, K, 9, distinct=False)
    lay = Layer(mq.Q4_K, mq.Q4_K, E, F, K, seed=80)
    Y = lay.run(X, ids, wts)
    pick = [0, M - 1]    # two tokens against the oracle (decoding is slow on the CPU)
    ref, bound = oracle.moe_ffn(lay.raw[0], lay.raw[1], lay.gu, lay.raw[2], lay.down, X[pick], ids[pick], wts[pick], E, F)
    say(f"moe phases M={M} k={k}: worst {float((np.abs(Y[pick] - ref) / bound).max()):.3f}")
    assert np.all(np.abs(Y[pick] - ref) <= bound)


@pytest.mark.parametrize("M", [2, 50])
def test_invalid_ids_add_nothing(M):
    E, F, K = 6, 256, 256
    X, ids, wts = inputs(M, 3, E, K, 10)
    ids[0] = -1                     # a token that no expert of this layer serves
    ids[1, 1] = E
    ids[M - 1, 2] = -2147483648
    wts[0] = np.nan                 # weights of dropped choices are not read into the sum
    res = np.random.default_rng(4).standard_normal((M, K)).astype(np.float32)
    lay = Layer(mq.Q4_K, mq.Q4_K, E, F, K, seed=90)
    Y = lay.check(X, ids, wts, residual=res)
    assert np.array_equal(Y[0], res[0])
    Y = lay.check(X, ids, wts)
    assert np.all(Y[0] == 0)
    ids[:] = 77
    assert np.array_equal(lay.run(X, ids, wts, residual=res), res)


@pytest.mark.parametrize("M", [1, 6, 33])
def test_repeated_expert_and_zero_weight(M):
    E, F, K = 3, 256, 512
    X, ids, wts = inputs(M, 4, E, K, 12, distinct=False)
    ids[0] = [1, 1, 2, 1]
    wts[0] = [0.5, 0.25, 0.0, -1.0]
    Layer(mq.Q6_K, mq.Q8_0, E, F, K, seed=100).check(X, ids, wts)


@pytest.mark.parametrize("M", [2, 8, 40])
def test_rows_do_not_depend_on_the_batch(M):
    """A token's bits are the same alone among other tokens of the same kernels."""
    E, F, K = 8, 512, 768
    lay = Layer(mq.Q4_K, mq.Q6_K, E, F, K, seed=110)
    X, ids, wts = inputs(M, 2, E, K, 13)
    Y = lay.run(X, ids, wts)
    perm = np.random.default_rng(1).permutation(M)
    assert np.array_equal(lay.run(X[perm], ids[perm], wts[perm]), Y[perm])
    ids2 = ids.copy()
    ids2[1:] = (ids2[1:] + 3) % E
    assert np.array_equal(lay.run(X, ids2, wts)[0], Y[0])
    assert np.array_equal(lay.run(X, ids, wts), Y)


def test_one_token_takes_many_choices():
    """More choices than waves, repeated experts, and the switch to the other kernels past 64."""
    E, F, K = 40, 256, 512
    lay = Layer(mq.Q4_K, mq.Q8_0, E, F, K, seed=115)
    for k in (16, 33, 64, 65, 200):
        X, ids, wts = inputs(1, k, E, K, k, distinct=False)
        ids[0, 1] = -1
        lay.check(X, ids, wts, what=f"k={k}")


@pytest.mark.parametrize("M", [4, 40])
def test_non_finite_tokens_stay_apart(M):
    E, F, K = 4, 256, 256
    lay = Layer(mq.Q4_K, mq.Q5_K, E, F, K, seed=120)
    X, ids, wts = inputs(M, 2, E, K, 15)
    Y = lay.run(X, ids, wts)
    Xb = X.copy()
    Xb[1, 5] = np.inf
    Xb[2, 200] = np.nan
    Xb[3, 0] = -np.inf
    Yb = lay.run(Xb, ids, wts)
    assert np.all(np.isnan(Yb[1:4]))
    rest = [0] + list(range(4, M))
    assert np.array_equal(Yb[rest], Y[rest])


def test_zero_tiny_and_large_activations():
    E, F, K = 4, 256, 512
    lay = Layer(mq.Q4_K, mq.Q4_K, E, F, K, seed=130)
    X, ids, wts = inputs(5, 2, E, K, 16)
    X[0] = 0
    X[1, :256] = 0
    X[2] *= 1e-25
    X[3] *= 1e4
    X[4, 7] = 1e6      # one value far above its block
    Y = lay.check(X, ids, wts)
    assert np.all(Y[0] == 0)


@pytest.mark.parametrize("M", [3, 36])
def test_output_may_be_input_or_residual(M):
    import torch
    E, F, K = 4, 256, 512
    lay = Layer(mq.Q4_K, mq.Q4_K, E, F, K, seed=140)
    X, ids, wts = inputs(M, 2, E, K, 17)
    res = np.random.default_rng(5).standard_normal((M, K)).astype(np.float32)
    ref = lay.run(X, ids, wts, residual=res)
    buf = to_dev(res, lay.dev)
    args = (lay.W[0], lay.W[1], lay.gu, lay.W[2], lay.down)
    mq.moe_ffn(*args, to_dev(X, lay.dev), to_dev(ids, lay.dev), to_dev(wts, lay.dev), E, F, residual=buf, Y=buf)
    torch.cuda.synchronize()
    assert np.array_equal(buf.cpu().numpy(), ref)
    x = to_dev(X, lay.dev)
    mq.moe_ffn(*args, x, to_dev(ids, lay.dev), to_dev(wts, lay.dev), E, F, residual=x, Y=x)
    torch.cuda.synchronize()
    assert np.array_equal(x.cpu().numpy(), lay.run(X, ids, wts, residual=X))


@pytest.mark.parametrize("qtype", [mq.Q8_0, mq.Q6_K], ids=["q8_0", "q6_K"])
@pytest.mark.parametrize("M", [1, 17])
def test_repacked_layouts_give_the_same_bits(qtype, M):
    E, F, K = 4, 256, 512
    lay = Layer(qtype, qtype, E, F, K, seed=150)
    X, ids, wts = inputs(M, 2, E, K, 18)
    Y = lay.run(X, ids, wts)
    lay.W = [mq.repack(lay.W[0], qtype, E * F, K), mq.repack(lay.W[1], qtype, E * F, K), mq.repack(lay.W[2], qtype, E * K, F)]
    lay.gu = lay.down = qtype | mq.REPACKED
    assert np.array_equal(lay.run(X, ids, wts), Y)


def test_many_experts_and_pairs():
    E, F, K = 512, 32, 64
    lay = Layer(mq.Q4_0, mq.Q8_0, E, F, K, seed=160)
    X, ids, wts = inputs(512, 8, E, K, 19)          # 4096 pairs
    ids[0, 0], ids[0, 1] = 511, 0
    lay.check(X, ids, wts)


def test_scratch_is_shared_by_shapes_and_needs_no_initial_value():
    import torch
    small = Layer(mq.Q4_K, mq.Q4_K, 4, 256, 256, seed=170)
    large = Layer(mq.Q8_0, mq.Q8_0, 4, 512, 1024, seed=171)
    a, b = inputs(2, 2, 4, 256, 20), inputs(40, 3, 4, 1024, 21)
    ra, rb = small.run(*a), large.run(*b)
    room = max(mq.moe_scratch_bytes(2, 2, 256, 256), mq.moe_scratch_bytes(40, 3, 512, 1024))
    scratch = torch.full((room,), 255, dtype=torch.uint8, device=small.dev)
    for _ in range(3):
        assert np.array_equal(small.run(*a, scratch=scratch), ra)
        assert np.array_equal(large.run(*b, scratch=scratch), rb)
