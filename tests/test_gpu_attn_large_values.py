"""mq_attn beside values whose scales are at f16's upper end: what a row does not see takes nothing from what it sees."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, Plan, attn_bound, bound_for, cache_on, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

KERNELS = ["attn_few", "attn_many"]
NORM = {mq.Q4_0: 1e-6, mq.Q8_0: 1.5e-6}       # as ordinary values are held to (test_gpu_attn.py)


def put(data, qtype, plan, heads, dim, b, pos, head, block, value):
    page, slot = ko.place(plan.table, plan.pages, plan.page, b, pos)
    s = ko.places(qtype, plan.page, dim)[5][slot, 32 * block]
    data.reshape(plan.pages, heads, -1)[page, head, s:s + 2] = np.frombuffer(np.float16(value).tobytes(), np.uint8)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("large", [300.0, 5000.0, -60000.0])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (256, 32)])
@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_do_not_see_a_large_value(qtype, large, dim, page, kernel):
    """A large block in a late token (the rows before it do not see it), in an early one behind a window, and in another head."""
    rng = np.random.default_rng([qtype, dim])
    heads, hq, n, window = 2, 6, 40, 50
    plan = Plan([n, n], [n + 300, n + 20], page, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    q = rng.standard_normal((plan.T, hq, dim)).astype(np.float32)
    bound = attn_bound(data, qtype, plan, heads, dim, q, dim ** -0.5)
    spots = [(0, n + 280, 0), (0, 30, 0), (0, n + 225, 1), (1, n + 19, 1)]       # sequence, position, head
    for i, (b, pos, head) in enumerate(spots):
        put(data, qtype, plan, heads, dim, b, pos, head, i % (dim // 32), large)
    dev = device()
    out = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev), window=window,
                  max_q=bound_for(kernel, plan, hq, heads), max_kv=plan.max_kv).cpu().numpy()
    assert mq.last_kernel() == kernel
    ref = ko.attn(data, qtype, plan.pages, page, heads, dim, plan.q_start, plan.kv_len, plan.table, q, dim ** -0.5, True, window)
    clear = np.ones((plan.T, heads), bool)
    for t, (b, pos) in enumerate(ko.rows_of(plan.q_start, plan.kv_len, plan.T)):
        for sb, at, head in spots:
            if sb == b and pos - window < at <= pos:
                clear[t, head] = False
    clear = np.repeat(clear, hq // heads, axis=1)
    assert 40 < clear.sum() < clear.size - 40
    err = np.abs(out - ref)
    ratio = float((err / bound)[clear].max())
    rel = float(np.linalg.norm(err[clear]) / np.linalg.norm(ref[clear]))
    print(f"  {ratio:.3f} of the bound, {rel:.2e} of the norm", flush=True)
    assert ratio <= 1.0 and rel <= NORM[qtype]
    # the others: a weight times a value to 2^-21, or to 2^-30 of the row's largest weight times the largest value, n of them over
    # the sum of weights (at most n largest ones: l >= 1)
    top = np.abs(ko.get(data, qtype, page, heads, dim)[1]).max()
    assert (err <= bound + 2.0 ** -20 * np.abs(ref).max((1, 2), keepdims=True) + window * 2.0 ** -30 * top).all()
    assert np.linalg.norm(err[~clear]) <= 2e-6 * np.linalg.norm(ref[~clear])


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kernel", KERNELS)
def test_every_value_is_large(qtype, n, dim, kernel):
    """Scales from 2^7 to f16's end in every block: each step has ordinary and large products, and NaN blocks beside them."""
    rng = np.random.default_rng([qtype, n, dim])
    heads, hq = 1, 4
    plan = Plan([n, n], [n + 200, n], 32, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    raw = data.reshape(plan.pages, heads, -1)
    for s in np.unique(ko.places(qtype, 32, dim)[5]):
        raw[:, :, s:s + 2] = (2.0 ** rng.uniform(7, 15.99, raw.shape[:2])).astype(np.float16)[..., None].view(np.uint8)
    q = rng.standard_normal((plan.T, hq, dim)).astype(np.float32)
    dev = device()

    def call():
        out = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev),
                      max_q=bound_for(kernel, plan, hq, heads), max_kv=plan.max_kv).cpu().numpy()
        assert mq.last_kernel() == kernel
        return out

    out = call()
    ref = ko.attn(data, qtype, plan.pages, 32, heads, dim, plan.q_start, plan.kv_len, plan.table, q, dim ** -0.5)
    assert np.linalg.norm(out - ref) <= NORM[qtype] * np.linalg.norm(ref)
    put(data, qtype, plan, heads, dim, 0, 40, 0, 1, np.nan)         # every row of the first sequence sees it, in its block
    got = call()
    assert np.isnan(got[:n, :, 32:64]).all()
    got[:n, :, 32:64] = out[:n, :, 32:64]
    assert np.array_equal(got, out)
