"""mq_attn where scores are large: one key takes nearly all of a row, up to f32's range.

A score is known to E: the roundings of q (2^-22), of the sums of codes with their offset (attn_bound), and of the score itself
and of the scale's product with log2 e (2^-22 of the row's largest score together).  Where E is small the bound is attn_bound's.
Elsewhere a key that is 2 E + 40 behind the largest score weighs less than e^-40: the row lies, in every dimension, between the
least and the largest value of the keys that are nearer (one key: it is that key's value), to 2^-20 of the largest value that
blocks of these scales hold."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, Plan, bound_for, cache_on, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

KERNELS = ["attn_few", "attn_many"]
SIZES = [0.1, 3.0, 30.0, 1e3, 1e5, 1e6, 3e6, 1e7, 2e7, 5e7, 1e8, 1e9, 1e12, 1e20, 1e30, 5e35]


def steps_of(data, qtype, plan, dim):
    raw = data.reshape(-1, ko.chunk_bytes(qtype, plan.page, dim))
    at = ko.places(qtype, plan.page, dim)
    s = np.unique(np.concatenate([at[4].ravel(), at[5].ravel()]))
    bits = raw[:, s].astype(np.uint16) | raw[:, s + 1].astype(np.uint16) << 8
    return float(np.abs(bits.view(np.float16).astype(np.float64)).max())


def check(out, data, qtype, plan, heads, dim, q, scale):
    C = 15 if qtype == mq.Q4_0 else 255
    step = steps_of(data, qtype, plan, dim)
    K, V = ko.get(data, qtype, plan.page, heads, dim)
    G = q.shape[1] // heads
    near_rows = 0
    for t, (b, pos) in enumerate(ko.rows_of(plan.q_start, plan.kv_len, plan.T)):
        spots = [ko.place(plan.table, plan.pages, plan.page, b, j) for j in range(pos + 1)]
        p, s = (np.array(a) for a in zip(*spots))
        for h in range(q.shape[1]):
            k, v = K[p, h // G, s], V[p, h // G, s]
            score = scale * (k @ q[t, h].astype(np.float64))
            E = abs(scale) * np.abs(q[t, h].astype(np.float64)).sum() * step * C * (2.0 ** -22 + (dim + 8) * 2.0 ** -24)
            E += 2.0 ** -22 * np.abs(score).max()
            got = out[t, h].astype(np.float64)
            if E < 0.05:
                e = np.exp(score - score.max())
                ref = (e / e.sum()) @ v
                limit = C / 2 * step * (np.expm1(2 * E) + 2.0 ** -21) + C * step * (2.0 ** -22 + (len(k) + 8) * 2.0 ** -24)
                assert np.abs(got - ref).max() <= limit, (t, h, np.abs(got - ref).max(), limit)
                continue
            near = score >= score.max() - 2 * E - 40
            near_rows += near.sum() == 1
            lo, hi = v[near].min(0), v[near].max(0)
            tol = 2.0 ** -20 * C * step
            assert (got >= lo - tol).all() and (got <= hi + tol).all(), (t, h, near.sum(), np.maximum(lo - got, got - hi).max(), tol)
    return near_rows


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("kv", [40, 2700])
@pytest.mark.parametrize("scale", [0.125, -1.0])
@pytest.mark.parametrize("kernel", KERNELS)
def test_scores_of_all_sizes(qtype, kv, scale, kernel):
    rng = np.random.default_rng([qtype, kv, int(scale > 0)])
    heads, dim, hq, n = 2, 64, 4, len(SIZES)
    plan = Plan([n, n], [kv, n + 3], 32, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    q = (np.tile(np.array(SIZES), 2)[:, None, None] * rng.standard_normal((plan.T, hq, dim))).astype(np.float32)
    q[:, 1] = q[::-1, 1]           # (rows of a tile with other sizes in another order)
    dev = device()
    out = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev), scale=scale,
                  max_q=bound_for(kernel, plan, hq, heads), max_kv=kv).cpu().numpy()
    assert mq.last_kernel() == kernel
    near = check(out, data, qtype, plan, heads, dim, q, scale)
    assert near >= 8       # rows that are one key's value


@pytest.mark.parametrize("kernel", KERNELS)
def test_rising_and_falling_scores(kernel):
    """Keys in order of their scores, rising and falling over several pieces: the running maximum moves at every step, or never."""
    rng = np.random.default_rng(5)
    dim, n = 64, 2
    plan = Plan([n, n], [2000, 2000], 32, rng)
    data = random_cache(mq.Q8_0, plan, 1, dim, rng)
    raw = data.reshape(plan.pages, 1, -1)
    at = ko.places(mq.Q8_0, 32, dim)
    for b in range(2):
        for j in range(2000):
            page, slot = ko.place(plan.table, plan.pages, 32, b, j)
            raw[page, 0, at[0][slot]] = 255                          # code 127
            s = np.unique(at[4][slot])
            size = 1e-5 * (1 + (j if b == 0 else 1999 - j))
            for i in s:
                raw[page, 0, i:i + 2] = np.frombuffer(np.float16(size).tobytes(), np.uint8)
    dev = device()
    for size in (1.0, 100.0, 1e4, 1e9, 1e30):
        q = np.full((plan.T, 3, dim), size, np.float32)
        out = mq.attn(cache_on(dev, data, mq.Q8_0, plan, 1, dim), plan.seqs(dev), to_dev(q, dev), scale=1.0,
                      max_q=bound_for(kernel, plan, 3, 1), max_kv=2000).cpu().numpy()
        assert mq.last_kernel() == kernel
        check(out, data, mq.Q8_0, plan, 1, dim, q, 1.0)


def one_sided(plan, heads, dim, rng):
    """A cache of 8 bits whose keys have no value below 1/8 (so that a query's sign is its scores' sign)."""
    data = random_cache(mq.Q8_0, plan, heads, dim, rng)
    raw = data.reshape(plan.pages, heads, -1)
    at = ko.places(mq.Q8_0, plan.page, dim)
    size = plan.page * dim
    raw[:, :, :size] = rng.integers(144, 256, raw[:, :, :size].shape)           # codes 16 to 127
    for s in np.unique(at[4]):
        raw[:, :, s:s + 2] = np.frombuffer(np.float16(2.0 ** -7).tobytes(), np.uint8)
    return data


@pytest.mark.parametrize("kv", [40, 2700])
@pytest.mark.parametrize("kernel", KERNELS)
def test_scores_past_the_range(kernel, kv):
    """Rows whose largest score passes f32's range, to either side, are NaN; beside a larger score that does not, one below the
    range weighs nothing; and other rows keep their bits."""
    rng = np.random.default_rng(kv)
    heads, dim, hq, n = 1, 64, 3, 6
    plan = Plan([n, n], [kv, n + 3], 32, rng)
    data = one_sided(plan, heads, dim, rng)
    raw = data.reshape(plan.pages, heads, -1)
    at = ko.places(mq.Q8_0, 32, dim)
    # the second sequence's third key is small: a thousandth of the least of the others
    page, slot = ko.place(plan.table, plan.pages, 32, 1, 2)
    raw[page, 0, at[0][slot]] = 129
    for s in np.unique(at[4][slot]):
        raw[page, 0, s:s + 2] = np.frombuffer(np.float16(2.0 ** -14).tobytes(), np.uint8)
    dev = device()

    def call(q, scale):
        out = mq.attn(cache_on(dev, data, mq.Q8_0, plan, heads, dim), plan.seqs(dev), to_dev(q, dev), scale=scale,
                      max_q=bound_for(kernel, plan, hq, heads), max_kv=kv).cpu().numpy()
        assert mq.last_kernel() == kernel
        return out

    base = np.abs(rng.standard_normal((plan.T, hq, dim))).astype(np.float32) + 0.5
    clean = call(base, 1.0)
    V = ko.get(data, mq.Q8_0, plan.page, heads, dim)[1]
    small = V[page, 0, slot]
    for sign in (1.0, -1.0):
        # a score is at least 64 * 0.5 * 2^38 * 2^-3 * 2^100 = 2^140 in magnitude, of the small key at most 64 * 8 * 2^138 * 2^-14 = 2^133
        q = base.copy()
        rows = np.zeros((plan.T, hq), bool)
        rows[1, 0] = rows[n - 1, 2] = rows[n, 1] = rows[n + 4, 0] = True
        q[rows] *= np.float32(sign * 2.0 ** 38)
        got = call(q, 2.0 ** 100)
        want = call(base, 2.0 ** 100)          # (scores of 2^102 and more: in range)
        assert np.isfinite(want).all()
        assert np.isnan(got[rows]).all(), (sign, np.argwhere(~np.isnan(got)).shape)
        assert np.array_equal(got[~rows], want[~rows])
    # the small key's score is in range, at least 2^20 above the others', which are below it
    q = base.copy()
    q[n:] *= np.float32(-2.0 ** 26)
    got = call(q, 2.0 ** 100)
    assert np.array_equal(got[:n], want[:n])
    tol = 2.0 ** -20 * np.abs(V).max()
    assert np.abs(got[n:] - small).max() <= tol
    assert np.array_equal(call(base, 1.0), clean)


@pytest.mark.parametrize("size,scale", [(1e-38, 3e38), (1e-38, 2e37), (3e-42, -3.4e38), (1e38, 1e-38), (1e37, 2e-38), (1e30, -1e-30)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_scales_over_their_range(size, scale, kernel):
    """Ordinary scores of tiny queries by large scales, and the other way round.  (A scale below f32's normal range: its own
    rounding, 2^-126 / 2^-149 at 1e-38, is in the f32 number that the oracle is given, too.)"""
    rng = np.random.default_rng(3)
    plan = Plan([2, 5], [300, 40], 32, rng)
    data = random_cache(mq.Q4_0, plan, 2, 64, rng)
    q = (size * 0.125 * rng.standard_normal((plan.T, 4, 64))).astype(np.float32)
    scale = float(np.float32(scale))
    dev = device()
    out = mq.attn(cache_on(dev, data, mq.Q4_0, plan, 2, 64), plan.seqs(dev), to_dev(q, dev), scale=scale,
                  max_q=bound_for(kernel, plan, 4, 2), max_kv=300).cpu().numpy()
    assert mq.last_kernel() == kernel
    check(out, data, mq.Q4_0, plan, 2, 64, q, scale)


@pytest.mark.parametrize("kernel", KERNELS)
def test_a_query_and_a_scale_at_their_ends(kernel):
    """|scale| times the row's largest value past f32's range: NaN either side; a row of zeros is the mean of its values."""
    rng = np.random.default_rng(9)
    plan = Plan([3, 3], [300, 40], 32, rng)
    data = one_sided(plan, 1, 64, rng)
    q = np.full((plan.T, 3, 64), 1e38, np.float32)
    q[:, 1] *= -1
    q[:, 2] = 0
    dev = device()
    for scale in (3e38, -3e38):
        out = mq.attn(cache_on(dev, data, mq.Q8_0, plan, 1, 64), plan.seqs(dev), to_dev(q, dev), scale=scale,
                      max_q=bound_for(kernel, plan, 3, 1), max_kv=300).cpu().numpy()
        assert mq.last_kernel() == kernel
        assert np.isnan(out[:, :2]).all()
        check(out[:, 2:], data, mq.Q8_0, plan, 1, 64, q[:, 2:], scale)
