"""mq_attn against the oracle in f64."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, Plan, attn_bound, bound_for, cache_on, check_attn, device, random_cache, to_dev

pytestmark = pytest.mark.gpu
KERNELS = ["attn_few", "attn_many"]

# f32 sums of codes with their offset: errors of a few half steps of 2^-24 beside values that the offset makes twice
# (8 bits: three times) as large, random over the 64 to 256 products and the 4 score blocks of a dimension of 128
NORM = {mq.Q4_0: 1e-6, mq.Q8_0: 1.5e-6}


def run(qtype, plan, hq, heads, dim, rng, causal=True, window=0, data=None, q=None, scale=None, what="", norm=True, scratch=None,
        kernel="attn_few", **kw):
    import torch
    dev = device()
    data = random_cache(qtype, plan, heads, dim, rng) if data is None else data
    q = rng.standard_normal((plan.T, hq, dim)).astype(np.float32) if q is None else q
    cache, seqs = cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev)
    out = torch.full((plan.T, hq, dim), 777.0, device=dev)
    args = dict(causal=causal, window=window, max_q=bound_for(kernel, plan, hq, heads), max_kv=plan.max_kv, scale=scale)
    args.update(kw)
    got = mq.attn(cache, seqs, to_dev(q, dev), out=out, scratch=scratch, **args)
    assert got is out and mq.last_kernel() == kernel
    out = out.cpu().numpy()
    scale = dim ** -0.5 if scale is None else scale
    ref = ko.attn(data, qtype, plan.pages, plan.page, heads, dim, plan.q_start, plan.kv_len, plan.table, q, scale, causal, window)
    check_attn(out, ref, attn_bound(data, qtype, plan, heads, dim, q, scale), what or f"{NAME[qtype]} {hq}/{heads}x{dim}",
               NORM[qtype] if norm else None)
    assert (out[np.isnan(ref)] == 777.0).all()
    return out


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("hq,heads,dim,page", [(14, 2, 64, 16), (7, 1, 128, 64), (2, 2, 256, 32), (32, 1, 128, 256), (5, 5, 64, 16)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 37), (False, 0)])
def test_one_row_of_each_sequence(qtype, hq, heads, dim, page, causal, window):
    rng = np.random.default_rng([qtype, hq, dim, page, window, causal])
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129, 257, 511, 700, 0]
    run(qtype, Plan([1 if l else 0 for l in kv], kv, page, rng, behind=1), hq, heads, dim, rng, causal, window)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("hq,heads,dim,page", [(14, 2, 64, 16), (7, 1, 128, 64), (4, 2, 256, 128), (3, 3, 128, 32)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_many_rows(qtype, hq, heads, dim, page, causal, window, kernel):
    rng = np.random.default_rng([qtype, hq, dim, page, window, causal, 1])
    plan = Plan([2, 0, 33, 5, 71], [9, 50, 33, 130, 171], page, rng, behind=3)
    run(qtype, plan, hq, heads, dim, rng, causal, window, kernel=kernel)


@pytest.mark.parametrize("window", [0, 1, 2, 16, 31, 1000])
@pytest.mark.parametrize("n", [1, 9, 40])
@pytest.mark.parametrize("kernel", KERNELS)
def test_windows(n, window, kernel):
    rng = np.random.default_rng([window, n])
    run(mq.Q4_0, Plan([n, n], [n, 999], 16, rng), 4, 1, 128, rng, True, window, kernel=kernel)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("hq,heads,dim,n,kv", [(28, 4, 128, 1, 5000), (14, 2, 64, 1, 9001), (8, 1, 256, 2, 3333), (16, 1, 128, 40, 2600), (2, 2, 256, 33, 1500)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_long_contexts(qtype, hq, heads, dim, n, kv, kernel):
    """Contexts that are cut over workgroups, beside a short sequence."""
    rng = np.random.default_rng([qtype, kv])
    run(qtype, Plan([n, 1], [kv, 3], 64, rng), hq, heads, dim, rng, kernel=kernel)


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_see_nothing(kernel):
    """Lengths of zero, lengths below the number of rows, pages that are not there."""
    rng = np.random.default_rng(1)
    plan = Plan([1, 6, 3, 4, 2], [0, 2, 40, 64, 20], 16, rng)
    plan.table[2] = -1                             # no page of the sequence is there
    plan.table[3, 1], plan.table[3, 3] = plan.pages, -2147483648
    out = run(mq.Q4_0, plan, 4, 2, 128, rng, what="empty rows", kernel=kernel)
    assert (out[:5] == 0).all() and (out[7:10] == 0).all()
    run(mq.Q8_0, plan, 4, 2, 64, rng, window=8, what="empty rows, window", kernel=kernel)
    run(mq.Q4_0, plan, 4, 2, 64, rng, causal=False, what="empty rows, not causal", kernel=kernel)


@pytest.mark.parametrize("n", [1, 20])
def test_lengths_past_the_bounds(n):
    """A length above the table's room uses what the table has; above max_kv it counts as max_kv."""
    rng = np.random.default_rng(2)
    plan = Plan([n, n], [90, 45], 16, rng, wide=0)
    plan.kv_len[0] = 16 * plan.width + 3
    run(mq.Q4_0, plan, 4, 2, 64, rng, what="past the table", max_kv=1000)
    plan.kv_len[0] = 90
    data, q = random_cache(mq.Q4_0, plan, 2, 64, rng), rng.standard_normal((plan.T, 4, 64)).astype(np.float32)
    dev = device()
    cache, seqs = cache_on(dev, data, mq.Q4_0, plan, 2, 64), plan.seqs(dev)
    short = mq.attn(cache, seqs, to_dev(q, dev), causal=False, max_q=n, max_kv=50).cpu().numpy()
    plan.kv_len[0] = 50
    ref = ko.attn(data, mq.Q4_0, plan.pages, 16, 2, 64, plan.q_start, plan.kv_len, plan.table, q, 64 ** -0.5, False)
    check_attn(short, ref, attn_bound(data, mq.Q4_0, plan, 2, 64, q, 64 ** -0.5), "max_kv")


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("kernel", KERNELS)
def test_what_no_length_covers_is_never_used(qtype, n, kernel):
    """NaN scales in every place behind a sequence's end, in unused pages and in masked keys."""
    rng = np.random.default_rng([qtype, n])
    heads, dim = 2, 128
    plan = Plan([n, n, 1], [n + 30, n, 77], 32, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    at = ko.places(qtype, plan.page, dim)
    chunk = ko.chunk_bytes(qtype, plan.page, dim)
    used = np.zeros((plan.pages, plan.page), bool)
    for b, l in enumerate(plan.kv):
        for j in range(l):
            used[plan.table[b, j // plan.page], j % plan.page] = True
    raw = data.reshape(plan.pages, heads, chunk)
    for which in (4, 5):
        for p, t in np.argwhere(~used):
            for s in np.unique(at[which][t]):
                raw[p, :, s:s + 2] = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)
    clean = data.copy().reshape(raw.shape)
    for which in (4, 5):
        for p, t in np.argwhere(~used):
            for s in np.unique(at[which][t]):
                clean[p, :, s:s + 2] = 0
    q = rng.standard_normal((plan.T, 6, dim)).astype(np.float32)
    a = run(qtype, plan, 6, heads, dim, rng, data=clean.reshape(-1), q=q, kernel=kernel)
    dev = device()
    b = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev),
                max_q=bound_for(kernel, plan, 6, heads), max_kv=plan.max_kv)
    assert mq.last_kernel() == kernel
    assert np.array_equal(a, b.cpu().numpy())


@pytest.mark.parametrize("n", [1, 24])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_bad_query_or_key_spoils_its_own_rows_only(n, bad, kernel):
    rng = np.random.default_rng(n)
    heads, dim, hq = 2, 64, 6
    plan = Plan([n, n], [n + 40, n + 3], 16, rng)
    data = random_cache(mq.Q4_0, plan, heads, dim, rng)
    q = rng.standard_normal((plan.T, hq, dim)).astype(np.float32)
    clean = run(mq.Q4_0, plan, hq, heads, dim, rng, data=data, q=q, kernel=kernel)
    qb = q.copy()
    qb[0, 1, 5] = bad
    dev = device()

    def call(data, q):
        return mq.attn(cache_on(dev, data, mq.Q4_0, plan, heads, dim), plan.seqs(dev), to_dev(q, dev),
                       max_q=bound_for(kernel, plan, hq, heads), max_kv=plan.max_kv).cpu().numpy()

    got = call(data, qb)
    assert np.isnan(got[0, 1]).all()
    got[0, 1] = clean[0, 1]
    assert np.array_equal(got, clean)
    if np.isnan(bad):       # a NaN block of a key, and one of a value, of the last token of the second sequence
        for which in (4, 5):
            raw = data.copy().reshape(plan.pages, heads, -1)
            page, slot = ko.place(plan.table, plan.pages, 16, 1, n + 2)
            s = ko.places(mq.Q4_0, 16, dim)[which][slot, 33]
            raw[page, 0, s:s + 2] = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)
            got = call(raw.reshape(-1), q)
            spoilt = got[-1, :3] if which == 4 else got[-1, :3, 32:]
            assert np.isnan(spoilt).all()
            spoilt[:] = (clean[-1, :3] if which == 4 else clean[-1, :3, 32:])
            assert np.array_equal(got, clean), which


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 30.0, 1e4])
@pytest.mark.parametrize("scale", [0.125, -0.2, 0.0, 1e-3])
@pytest.mark.parametrize("kernel", KERNELS)
def test_ranges_of_queries(size, scale, kernel):
    """Scores from nothing to one key taking all, a negative scale, and zero: the mean."""
    rng = np.random.default_rng(11)
    plan = Plan([3, 18], [70, 200], 32, rng)
    q = (size * rng.standard_normal((plan.T, 4, 64))).astype(np.float32)
    q[1] = 0.0
    q[:, 1, ::2] *= 1e-5
    big = size * abs(scale) * 64 > 100
    import torch
    if big:       # one key takes all where the others are exp(-bound) behind: compared where the gap is clear
        dev = device()
        data = random_cache(mq.Q4_0, plan, 2, 64, rng)
        out = mq.attn(cache_on(dev, data, mq.Q4_0, plan, 2, 64), plan.seqs(dev), to_dev(q, dev), scale=scale,
                      max_q=bound_for(kernel, plan, 4, 2), max_kv=200).cpu().numpy()
        ref = ko.attn(data, mq.Q4_0, plan.pages, 32, 2, 64, plan.q_start, plan.kv_len, plan.table, q, scale)
        assert torch.isfinite(torch.from_numpy(out)).all()
        assert np.mean(np.abs(out - ref).max(-1) < 1e-2) > 0.9
    else:
        run(mq.Q4_0, plan, 4, 2, 64, rng, q=q, scale=scale, norm=False, kernel=kernel)


@pytest.mark.parametrize("n", [1, 17])
def test_strided_queries_and_large_bounds(n):
    """Queries that are parts of a product's rows; bounds far above the lengths."""
    import torch
    dev = device()
    rng = np.random.default_rng(12)
    plan = Plan([n, 2 * n], [40, 300], 16, rng)
    data = random_cache(mq.Q4_0, plan, 2, 128, rng)
    x = rng.standard_normal((plan.T, 10, 128)).astype(np.float32)
    xd = to_dev(x, dev)
    cache, seqs = cache_on(dev, data, mq.Q4_0, plan, 2, 128), plan.seqs(dev)
    ref = ko.attn(data, mq.Q4_0, plan.pages, 16, 2, 128, plan.q_start, plan.kv_len, plan.table, x[:, 2:8], 128 ** -0.5)
    bound = attn_bound(data, mq.Q4_0, plan, 2, 128, x, 128 ** -0.5)
    for max_q, max_kv in ((2 * n, 300), (500, 1 << 17), (5000, 400), (None, None)):
        got = mq.attn(cache, seqs, xd[:, 2:8], max_q=max_q, max_kv=max_kv)
        torch.cuda.synchronize()
        check_attn(got.cpu().numpy(), ref, bound, f"max_q={max_q} max_kv={max_kv}", 1e-6)


def test_rows_past_max_q_are_left():
    import torch
    dev = device()
    rng = np.random.default_rng(13)
    plan = Plan([20, 3], [25, 30], 16, rng)
    data = random_cache(mq.Q4_0, plan, 1, 64, rng)
    q = rng.standard_normal((plan.T, 3, 64)).astype(np.float32)
    cache, seqs = cache_on(dev, data, mq.Q4_0, plan, 1, 64), plan.seqs(dev)
    whole = mq.attn(cache, seqs, to_dev(q, dev), max_q=20, max_kv=30).cpu()
    out = torch.full((plan.T, 3, 64), 777.0, device=dev)
    mq.attn(cache, seqs, to_dev(q, dev), max_q=7, max_kv=30, out=out)
    out = out.cpu()
    assert (out[7:20] == 777.0).all()
    assert torch.allclose(out[:7], whole[:7], rtol=0, atol=1e-5) and torch.allclose(out[20:], whole[20:], rtol=0, atol=1e-5)


def test_a_cache_of_more_than_four_gib():
    import torch
    dev = device()
    rng = np.random.default_rng(14)
    heads, dim, page = 8, 128, 256
    small = Plan([1, 30], [600, 200], page, rng)
    data = random_cache(mq.Q4_0, small, heads, dim, rng)
    chunk = heads * ko.chunk_bytes(mq.Q4_0, page, dim)
    pages = (5 << 30) // chunk
    big = torch.zeros(pages * chunk, dtype=torch.uint8, device=dev)
    big[-small.pages * chunk:] = to_dev(data, dev)
    q = to_dev(rng.standard_normal((31, 16, dim)).astype(np.float32), dev)
    ref = mq.attn(cache_on(dev, data, mq.Q4_0, small, heads, dim), small.seqs(dev), q, max_q=30, max_kv=600)
    small.table = np.where(small.table >= 0, small.table + pages - small.pages, -1).astype(np.int32)
    got = mq.attn(mq.KVCache(big, mq.Q4_0, pages, page, heads, dim), small.seqs(dev), q, max_q=30, max_kv=600)
    torch.cuda.synchronize()
    assert torch.equal(ref, got)


@pytest.mark.parametrize("kernel", KERNELS)
def test_the_same_bits_every_time(kernel):
    """Results do not depend on which workgroup ends last, nor on what a workspace held (its counters aside)."""
    import torch
    dev = device()
    rng = np.random.default_rng(15)
    plan = Plan([1, 1, 2], [4000, 1500, 3], 64, rng)
    data = random_cache(mq.Q4_0, plan, 4, 128, rng)
    q = to_dev(rng.standard_normal((plan.T, 28, 128)).astype(np.float32), dev)
    cache, seqs = cache_on(dev, data, mq.Q4_0, plan, 4, 128), plan.seqs(dev)
    max_q = bound_for(kernel, plan, 28, 4)
    need = mq.attn_scratch_bytes(mq.Q4_0, 3, 28, 4, 128, max_q, 4000)
    assert need > 1 << 18        # joined pieces
    first = None
    for fill in (0, 255, 17):
        scratch = torch.full((need,), fill, dtype=torch.uint8, device=dev)
        scratch[:1 << 18] = 0
        for _ in range(5):
            out = mq.attn(cache, seqs, q, max_q=max_q, max_kv=4000, scratch=scratch)
            first = out if first is None else first
            assert torch.equal(first, out)
        assert int(scratch[:1 << 18].sum()) == 0


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("n", [1, 9, 40])
@pytest.mark.parametrize("large", [200.0, 300.0, 5000.0, 60000.0, -60000.0])
@pytest.mark.parametrize("kernel", KERNELS)
def test_values_of_all_sizes(qtype, n, large, kernel):
    """Scales of single blocks far above and below the others', in the middle of a context and at its end: f16's whole range.
    Errors to 2^-16 beside those of the largest values (which are held to 22 bits, as the small ones are without them)."""
    rng = np.random.default_rng([qtype, n])
    heads, dim = 2, 128
    plan = Plan([n, n], [n + 260, n + 40], 32, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    raw = data.reshape(plan.pages, heads, -1)
    at = ko.places(qtype, plan.page, dim)[5]

    def put(b, pos, block, value):
        page, slot = ko.place(plan.table, plan.pages, plan.page, b, pos)
        s = at[slot, 32 * block]
        raw[page, :, s:s + 2] = np.frombuffer(np.float16(value).tobytes(), np.uint8)

    put(0, 100, 1, large)
    put(0, n + 259, 3, large / 7)
    put(0, 0, 0, 1e-6)
    put(1, 3, 2, 6e-8)
    put(1, n + 39, 0, large)         # seen by the last row alone
    q = rng.standard_normal((plan.T, 6, dim)).astype(np.float32)
    dev = device()
    out = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev),
                  max_q=bound_for(kernel, plan, 6, heads), max_kv=plan.max_kv).cpu().numpy()
    assert mq.last_kernel() == kernel
    ref = ko.attn(data, qtype, plan.pages, plan.page, heads, dim, plan.q_start, plan.kv_len, plan.table, q, dim ** -0.5)
    err = np.abs(out - ref)
    # by rows: those that see a large value, and those of the second sequence that do not
    big = np.abs(ref).max((1, 2))[:, None, None]
    assert (err <= 2.0 ** -16 + 2.0 ** -18 * big).all(), float((err / (2.0 ** -16 + 2.0 ** -18 * big)).max())
    assert np.linalg.norm(err[:n]) <= 2e-6 * np.linalg.norm(ref[:n])


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("unit", [1e-5, 1e-3, 50.0])
@pytest.mark.parametrize("kernel", KERNELS)
def test_values_all_small_or_large(n, unit, kernel):
    """Relative accuracy does not depend on the values' size (scales in f16's subnormal range are exact, too)."""
    rng = np.random.default_rng(n)
    plan = Plan([n, n], [n + 200, n], 16, rng)
    data = random_cache(mq.Q4_0, plan, 1, 64, rng)
    raw = data.reshape(plan.pages, 1, -1)
    vs = ko.places(mq.Q4_0, plan.page, 64)[5]
    for s in np.unique(vs):
        d = raw[:, :, s:s + 2].copy().view(np.float16).astype(np.float32) * (unit / 0.22)
        raw[:, :, s:s + 2] = d.astype(np.float16).view(np.uint8)
    q = rng.standard_normal((plan.T, 7, 64)).astype(np.float32)
    dev = device()
    out = mq.attn(cache_on(dev, data, mq.Q4_0, plan, 1, 64), plan.seqs(dev), to_dev(q, dev),
                  max_q=bound_for(kernel, plan, 7, 1), max_kv=n + 200).cpu().numpy()
    ref = ko.attn(data, mq.Q4_0, plan.pages, 16, 1, 64, plan.q_start, plan.kv_len, plan.table, q, 0.125)
    assert np.linalg.norm(out - ref) <= 1e-6 * np.linalg.norm(ref)
