"""mq_kv_append and mq_kv_read against the oracle: the cache byte for byte, the queries within one rounding."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, Plan, cache_on, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

ROPES = {0: mq.ROPE_NONE, 1: mq.ROPE_HALF, 2: mq.ROPE_INTERLEAVED}


def freqs(rot, base=10000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def expected(data, qtype, plan, heads, dim, q, k, v, qn, kn, eps, rope, f, pos=None):
    """(q out f64, NaN rows where nothing is written; the cache's bytes after the call)."""
    rows = ko.rows_of(plan.q_start, plan.kv_len, plan.T)
    at = np.array([p for _, p in rows]) if pos is None else pos
    qe = None if q is None else ko.rotated(ko.normed(q, qn, eps), at, f, rope)
    ke = ko.rotated(ko.normed(k, kn, eps), at, f, rope).astype(np.float32)
    data = data.copy()
    for t, (b, p) in enumerate(rows):
        if b < 0:
            if qe is not None:
                qe[t] = np.nan
            continue
        spot = ko.place(plan.table, plan.pages, plan.page, b, p)
        if spot is None:
            continue
        for h in range(heads):
            for which, x in ((0, ke), (1, v)):
                s, c = ko.quantize(x[t, h], qtype)
                ko.put(data, qtype, plan.page, heads, dim, *spot, h, which, s, c)
    return qe, data


def same_cache(got, want, qtype, plan, heads, dim):
    """Bytes equal, or (a scale that is a NaN) NaN at the same places."""
    diff = np.nonzero(got != want)[0]
    if len(diff) == 0:
        return True
    chunk = ko.chunk_bytes(qtype, plan.page, dim)
    row = 2 * plan.page * dim * ko.BITS[qtype] // 8
    for i in diff:
        off = i % chunk
        if off < row:
            return False
        j = i - (off - row) % 2
        a, b = (x[j:j + 2].view(np.float16)[0] for x in (got, want))
        if not (np.isnan(a) and np.isnan(b)):
            return False
    return True


def check(qtype, plan, hq, heads, dim, rng, rope=1, rot=None, norm=False, fused=False, pos=None, edit=None, eps=1e-6):
    import torch
    dev = device()
    rot = dim if rot is None else rot
    x = rng.standard_normal((plan.T, hq + 2 * heads, dim)).astype(np.float32)
    if edit:
        edit(x)
    qn, kn = ((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32) for _ in range(2)) if norm else (None, None)
    f = freqs(rot) if rope else None
    before = random_cache(qtype, plan, heads, dim, rng)
    q, k, v = x[:, :hq], x[:, hq:hq + heads], x[:, hq + heads:]
    if fused:
        xd = to_dev(x, dev)
        qd, kd, vd = xd[:, :hq], xd[:, hq:hq + heads], xd[:, hq + heads:]
    else:
        qd, kd, vd = (to_dev(a, dev) for a in (q, k, v))
    cache, seqs = cache_on(dev, before, qtype, plan, heads, dim), plan.seqs(dev)
    opt = lambda a: None if a is None else to_dev(a, dev)   # noqa: E731
    out = torch.full((plan.T, hq, dim), 777.0, device=dev)
    got = mq.kv_append(cache, seqs, kd, vd, q=qd, q_norm=opt(qn), k_norm=opt(kn), eps=eps, rope=ROPES[rope],
                       inv_freq=opt(f), pos=opt(pos), q_out=out)
    assert got is out and mq.last_kernel() == "kv_append"
    qe, data = expected(before, qtype, plan, heads, dim, q, k, v, qn, kn, eps, rope, f, pos)
    out, after = out.cpu().numpy(), cache.data.cpu().numpy()
    dead = np.isnan(qe).all((1, 2)) & (np.array([b for b, _ in ko.rows_of(plan.q_start, plan.kv_len, plan.T)]) < 0)
    assert (out[dead] == 777.0).all()
    live = ~dead
    # formed in f64 and rounded once: half a step of the value, and f64's own error of the largest factor
    tol = 2.0 ** -24 * np.abs(qe[live]) * (1 + 1e-6) + 1e-12 * np.nanmax(np.abs(x[live][:, :hq]), initial=1.0) + 2.0 ** -149
    ok = (np.abs(out[live] - qe[live]) <= tol) | (np.isnan(out[live]) & np.isnan(qe[live])) | (out[live] == qe[live].astype(np.float32))
    assert ok.all(), np.argwhere(~ok)[:5]
    assert same_cache(after, data, qtype, plan, heads, dim), "cache bytes"
    kr, vr = mq.kv_read(cache, seqs, plan.T, k=torch.full((plan.T, heads, dim), 777.0, device=dev))
    assert mq.last_kernel() == "kv_read"
    K, V = ko.get(data, qtype, plan.page, heads, dim)
    kr, vr = kr.cpu().numpy(), vr.cpu().numpy()
    for t, (b, p) in enumerate(ko.rows_of(plan.q_start, plan.kv_len, plan.T)):
        if b < 0:
            assert (kr[t] == 777.0).all()
            continue
        spot = ko.place(plan.table, plan.pages, plan.page, b, p)
        for r, whole in ((kr, K), (vr, V)):
            want = np.zeros((heads, dim)) if spot is None else whole[spot[0], :, spot[1]]
            assert np.array_equal(r[t], want.astype(np.float32), equal_nan=True)
    return out, after


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("hq,heads,dim,page", [(14, 2, 64, 16), (7, 1, 128, 64), (5, 5, 256, 32), (3, 1, 64, 256)])
@pytest.mark.parametrize("rope,norm,fused", [(1, True, False), (2, False, True), (0, True, True), (1, False, True)])
def test_append(qtype, hq, heads, dim, page, rope, norm, fused):
    rng = np.random.default_rng([qtype, hq, dim, page, rope, norm])
    plan = Plan([1, 0, 19, 3], [1, 40, 19 + page - 2, 300], page, rng, behind=2)
    check(qtype, plan, hq, heads, dim, rng, rope=rope, norm=norm, fused=fused)


@pytest.mark.parametrize("rot", [2, 34, 64, 96, 126])
@pytest.mark.parametrize("rope", [1, 2])
def test_part_of_a_head_is_rotated(rope, rot):
    rng = np.random.default_rng(rot + rope)
    check(mq.Q4_0, Plan([5, 2], [70, 2], 16, rng), 4, 2, 128, rng, rope=rope, rot=rot, norm=rot == 64)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
def test_far_positions(qtype):
    """Angles of up to 2^31 - 1, and below zero."""
    rng = np.random.default_rng(3)
    plan = Plan([6], [6], 16, rng)
    check(qtype, plan, 3, 1, 128, rng, pos=np.array([0, 1, -1, 1 << 20, (1 << 31) - 1, -(1 << 31)], np.int32))


def test_one_row_and_many_sequences():
    rng = np.random.default_rng(4)
    check(mq.Q4_0, Plan([1], [1], 64, rng), 28, 4, 128, rng, fused=True)
    n = [1, 0] * 70 + [2]       # more than a wave of sequences
    check(mq.Q4_0, Plan(n, [a + 20 for a in n], 16, rng), 2, 1, 64, rng)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
def test_special_values(qtype):
    def edit(x):
        x[0] = 0.0                                          # zero blocks
        x[1, :, ::3], x[1, :, 1::3] = 1e-38, -3e-39         # scales that vanish in f16
        x[2] *= 1e30                                        # and that pass it
        x[3, :, 5] = np.nan
        x[4, :, 40] = np.inf
        x[5] *= 2e4                                         # largest scales (8 bits), past them (4 bits: some)
        x[6] = np.where(np.arange(x.shape[-1]) % 2, 0.75, -0.75)   # ties of magnitude
        x[7] *= 1e-7                                        # subnormal scales
    rng = np.random.default_rng(6)
    for norm in (False, True):
        check(qtype, Plan([8], [8], 16, rng), 2, 2, 64, rng, rope=0, norm=norm, edit=edit)


@pytest.mark.parametrize("norm", [False, True])
def test_pages_that_are_not_there(norm):
    """Table entries outside the cache, positions past the table and below zero: q is served, nothing is written."""
    rng = np.random.default_rng(7)
    plan = Plan([4, 3, 2, 5], [34, 3, 60, 5], 16, rng, wide=0)
    plan.table[0, 2], plan.table[1, 0] = plan.pages, -7
    plan.kv_len[2] = 16 * plan.width + 2           # both rows past the table
    plan.kv_len[3] = 2                             # three of five rows before the first place
    check(mq.Q4_0, plan, 2, 2, 64, rng, norm=norm)


def test_in_place_and_without_queries():
    import torch
    dev = device()
    rng = np.random.default_rng(8)
    plan = Plan([3, 5], [10, 5], 16, rng)
    x = to_dev(rng.standard_normal((8, 8, 128)).astype(np.float32), dev)
    f = to_dev(freqs(128), dev)
    data = random_cache(mq.Q4_0, plan, 2, 128, rng)
    seqs = plan.seqs(dev)
    c0, c1, c2 = (cache_on(dev, data, mq.Q4_0, plan, 2, 128) for _ in range(3))
    ref = mq.kv_append(c0, seqs, x[:, 4:6], x[:, 6:], q=x[:, :4], inv_freq=f)
    assert mq.kv_append(c1, seqs, x[:, 4:6], x[:, 6:], inv_freq=f) is None
    y = x.clone()
    mq.kv_append(c2, seqs, y[:, 4:6], y[:, 6:], q=y[:, :4], q_out=y[:, :4], inv_freq=f)
    torch.cuda.synchronize()
    assert torch.equal(ref, y[:, :4]) and torch.equal(x[:, 4:], y[:, 4:])
    assert torch.equal(c0.data, c1.data) and torch.equal(c0.data, c2.data)


def test_a_place_behind_four_gib():
    import torch
    dev = device()
    rng = np.random.default_rng(9)
    heads, dim, page = 8, 128, 256
    pages = (5 << 30) // (heads * ko.chunk_bytes(mq.Q4_0, page, dim))
    cache = mq.KVCache(torch.zeros(mq.kv_cache_bytes(mq.Q4_0, pages, page, heads, dim), dtype=torch.uint8, device=dev),
                       mq.Q4_0, pages, page, heads, dim)
    seqs = mq.KVSeqs(*(torch.tensor(a, dtype=torch.int32, device=dev) for a in ([0, 2], [257], [[pages - 1, 0]])))
    k, v = (rng.standard_normal((2, heads, dim)).astype(np.float32) for _ in range(2))
    mq.kv_append(cache, seqs, to_dev(k, dev), to_dev(v, dev), rope=mq.ROPE_NONE)
    kr, vr = mq.kv_read(cache, seqs, 2)
    for got, x in ((kr, k), (vr, v)):
        assert np.array_equal(got.cpu().numpy(), ko.values(*ko.quantize(x, mq.Q4_0), mq.Q4_0).astype(np.float32))
    chunk = heads * ko.chunk_bytes(mq.Q4_0, page, dim)
    assert int((cache.data[chunk:-chunk] != 0).sum()) == 0
