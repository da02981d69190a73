"""mq_sample against the oracle, token by token: ids equal, probabilities within f32's rounding."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import device, to_dev

pytestmark = pytest.mark.gpu


def run(l, u, T=None, k=None, p=None, m=None, stride=None, scratch=None):
    import torch
    dev = device()
    M, V = l.shape
    ld = to_dev(l, dev)
    if stride:
        wide = torch.full((M, stride), 1e9, device=dev)
        wide[:, :V] = ld
        ld = wide[:, :V]
    opt = lambda a, t=np.float32: None if a is None else to_dev(np.asarray(a, t), dev)   # noqa: E731
    ids, probs = mq.sample(ld, to_dev(np.asarray(u, np.float32), dev), temperature=opt(T), top_k=opt(k, np.int32), top_p=opt(p),
                           min_p=opt(m), scratch=scratch)
    assert mq.last_kernel().startswith("sample")
    return ids.cpu().numpy(), probs.cpu().numpy()


def check(l, u, T=None, k=None, p=None, m=None, what="", **kw):
    ids, probs = run(l, u, T, k, p, m, **kw)
    f32 = lambda a, i: float(np.float32(a[i]))   # noqa: E731
    for i in range(len(l)):
        want, prob = ko.sample(l[i], f32(u, i), 1.0 if T is None else f32(T, i), 0 if k is None else int(k[i]),
                               1.0 if p is None else f32(p, i), 0.0 if m is None else f32(m, i))
        assert ids[i] == want, (what, i, ids[i], want)
        # one rounding to f32, and sums of at most 2^20 masses that are each within 2^-44
        assert abs(probs[i] - prob) <= 2.0 ** -24 * prob + 2.0 ** -23 * 2.0 ** -20 * prob + 1e-30, (what, i, probs[i], prob)


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 4097, 32003, 152064])
@pytest.mark.parametrize("M", [1, 5])
def test_every_filter(V, M):
    rng = np.random.default_rng([V, M])
    l = (2.5 * rng.standard_normal((M, V))).astype(np.float32)
    for T, k, p, m in ((None, None, None, None), (0.7, None, None, None), (None, 40, None, None), (None, None, 0.9, None),
                       (None, None, None, 0.1), (0.8, 50, 0.95, 0.02), (1.7, V - 1, 0.999, None), (None, 1, 0.5, None),
                       (0.01, None, 0.99, None), (5.0, 3, 0.3, 0.9)):
        full = lambda a: None if a is None else np.full(M, a)   # noqa: E731
        for u in (0.0, 0.37, 0.9999999):
            check(l, np.full(M, u) if u else rng.random(M), full(T), full(k), full(p), full(m), what=(V, T, k, p, m, u))


@pytest.mark.parametrize("V", [50, 3000, 40000])
def test_settings_of_each_row(V):
    rng = np.random.default_rng(V)
    M = 33
    l = (3 * rng.standard_normal((M, V))).astype(np.float32)
    l[rng.random(l.shape) < 0.3] = -np.inf
    l[rng.random(l.shape) < 0.01] = np.nan
    check(l, rng.random(M), T=np.where(rng.random(M) < 0.2, 0, 0.3 + rng.random(M)), k=rng.integers(-1, 200, M),
          p=rng.uniform(0.5, 1.1, M), m=rng.uniform(-0.1, 0.3, M), stride=V + 5)


@pytest.mark.parametrize("V", [70, 5000, 70001])
def test_equal_logits(V):
    """Ties go to the lower index; masses that end exactly at a border belong to the shorter prefix."""
    M = 12
    l = np.zeros((M, V), np.float32)
    l[6:, ::3] = 1.0
    l[8:, ::3] = 20.0
    l[10:, 1::2] = -0.0
    u = np.linspace(0, 0.999, M)
    check(l, u)
    check(l, u, k=np.arange(1, M + 1) * (V // 13))
    check(l, u, p=np.full(M, 0.5))
    check(l, u, p=np.full(M, 0.25), k=np.full(M, V // 2))
    check(l, u, T=np.full(M, 0.0))
    check(l, u, m=np.full(M, 1.0))


def test_rows_without_a_choice_and_infinities():
    V = 3000
    l = np.full((8, V), -np.inf, np.float32)
    l[1] = np.nan
    l[2, 77] = -5.0
    l[3, [5, 900]] = np.inf
    l[4, 3] = 3e38
    l[4, 4] = -3e38
    l[5, :] = -3.4e38
    l[6, 10:20] = np.nan
    l[6, 2999] = 1.0
    l[7, :] = np.linspace(-60, 0, V)
    for u in (0.0, 0.5, 0.99):
        for T in (None, np.full(8, 0.5), np.zeros(8), np.full(8, -1.0)):
            check(l, np.full(8, u), T=T, k=np.full(8, 3), p=np.full(8, 0.9))
            check(l, np.full(8, u), T=T)
            check(l, np.full(8, u), T=T, p=np.full(8, 0.7), m=np.full(8, 0.2))
    ids, probs = run(l, np.full(8, 0.3))
    assert ids[0] == ids[1] == -1 and probs[0] == probs[1] == 0


def test_settings_out_of_range():
    """top_p of zero and below keeps the first token, settings that are NaN keep all (a temperature: the first)."""
    rng = np.random.default_rng(5)
    l = rng.standard_normal((6, 500)).astype(np.float32)
    top = l.argmax(1)
    assert (run(l, np.full(6, 0.9), p=np.zeros(6))[0] == top).all() and (run(l, np.full(6, 0.9), p=np.full(6, -3.0))[0] == top).all()
    assert (run(l, np.full(6, 0.9), T=np.full(6, np.nan))[0] == top).all()
    ref = run(l, np.full(6, 0.7))[0]
    assert (run(l, np.full(6, 0.7), p=np.full(6, np.nan), m=np.full(6, np.nan), k=np.full(6, -9))[0] == ref).all()
    assert (run(l, np.full(6, 0.7), m=np.full(6, 7.0))[0] == top).all()
    last = [np.nonzero(np.isfinite(r))[0][-1] for r in l]
    assert (run(l, np.full(6, 1.0))[0] == last).all() and (run(l, np.full(6, 9.0))[0] == last).all()
    assert (run(l, np.full(6, -1.0))[0] == 0).all() and (run(l, np.full(6, np.nan))[0] == 0).all()


def test_many_rows_and_a_shared_workspace():
    import torch
    rng = np.random.default_rng(6)
    scratch = torch.zeros(max(mq.sample_scratch_bytes(300, 9000), 4 << 20), dtype=torch.uint8, device=device())
    for M, V in ((300, 700), (3, 9000), (70, 9000), (300, 9000), (1, 40)):
        l = (2 * rng.standard_normal((M, V))).astype(np.float32)
        check(l, rng.random(M), T=np.full(M, 0.9), k=rng.integers(0, 60, M), p=rng.uniform(0.6, 1.0, M), scratch=scratch)
        assert int(scratch[:4 << 20].sum()) == 0


def test_the_draws_follow_the_distribution():
    """Counts over an even grid of u are the probabilities to one draw a token."""
    rng = np.random.default_rng(7)
    V, M = 40, 4096
    row = (1.5 * rng.standard_normal(V)).astype(np.float32)
    ids, _ = run(np.tile(row, (M, 1)), (np.arange(M) + 0.5) / M)
    p = np.exp(row.astype(np.float64) - row.max())
    assert np.abs(np.bincount(ids, minlength=V) - M * p / p.sum()).max() <= 1.0
