"""Shared inputs and checks of the tests of the paged cache, the attention over it and sampling."""

import numpy as np

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from gpu_cases import device, to_dev

TYPES = [mq.Q4_0, mq.Q8_0]
NAME = {mq.Q4_0: "q4_0", mq.Q8_0: "q8_0"}


class Plan:
    """Sequences of n[b] rows that end a cache of kv[b] tokens, their pages in random order; pages past a
    sequence's end are -1 in the table."""

    def __init__(self, n, kv, page, rng, spare=3, wide=1, behind=0):
        self.n, self.kv, self.page = list(n), list(kv), page
        per = [-(-max(l, 0) // page) for l in kv]
        self.width, self.pages = max(per + [1]) + wide, sum(per) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(n), self.width), -1, np.int32)
        at = 0
        for b, p in enumerate(per):
            self.table[b, :p] = order[at:at + p]
            at += p
        self.q_start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.kv_len = np.array(kv, np.int32)
        self.T = int(sum(n)) + behind

    def seqs(self, dev):
        return mq.KVSeqs(*(to_dev(a, dev) for a in (self.q_start, self.kv_len, self.table)))

    @property
    def max_q(self):
        return max(max(self.n), 1)

    @property
    def max_kv(self):
        return max(max(self.kv), 1)


def bound_for(kernel, plan, hq, heads):
    """The bound max_q with which mq_attn takes the kernel: the lengths themselves, or the first bound above 256 rows and
    768 tiles of 16 (of the call's sequences and heads) that the kernel of many rows serves."""
    if kernel == "attn_few":
        return plan.max_q
    group = hq // heads
    tiles = 768 // (len(plan.n) * heads) + 1
    return max(16 * (tiles - 1) // group + 1, 256 // group + 1)


def random_cache(qtype, plan, heads, dim, rng, unit=None):
    """Bytes of a cache whose values have a deviation of about 1 (scales of both signs for 4 bits)."""
    chunk = ko.chunk_bytes(qtype, plan.page, dim)
    data = rng.integers(0 if qtype == mq.Q4_0 else 1, 256, (plan.pages, heads, chunk)).astype(np.uint8)
    count = 2 * plan.page * (dim // 32)
    d = (unit or (0.22 if qtype == mq.Q4_0 else 0.0136)) * (0.6 + 0.8 * rng.random((plan.pages, heads, count)))
    if qtype == mq.Q4_0:
        d *= np.where(rng.random(d.shape) < 0.5, -1, 1)
    data[:, :, chunk - 2 * count:] = d.astype(np.float16).view(np.uint8).reshape(plan.pages, heads, 2 * count)
    return data.reshape(-1)


def cache_on(dev, data, qtype, plan, heads, dim):
    return mq.KVCache(to_dev(data, dev), qtype, plan.pages, plan.page, heads, dim)


def attn_bound(data, qtype, plan, heads, dim, q, scale):
    """Largest error of an element of a row, [T, 1, 1] for finite inputs, from the roundings alone.

    A factor split into two f16 keeps it to 2^-22; a sum of n products in f32 errs by at most n 2^-24 of the sum
    of their magnitudes, where codes count with their offset (at most C = 15 or 255 steps of a block).  With
    s the largest score error so found, the weights err by a factor within exp(2 s) - 1 plus 2^-21 for exp and the
    running rescales, and the second sum by 2^-22 + n 2^-24 over at most n = kv keys of at most C steps."""
    at = ko.places(qtype, plan.page, dim)
    raw = data.reshape(plan.pages, heads, -1)
    step = 0.0
    for which in (4, 5):
        b = np.unique(at[which])
        bits = raw[:, :, b].astype(np.uint16) | (raw[:, :, b + 1].astype(np.uint16) << 8)
        step = max(step, float(np.nanmax(np.abs(bits.view(np.float16).astype(np.float64)))))
    C = 15 if qtype == mq.Q4_0 else 255
    s = abs(scale) * np.abs(q.astype(np.float64)).sum(-1).max(-1) * step * C * (2.0 ** -22 + (dim + 8) * 2.0 ** -24)
    top = C / 2 * step
    return (top * (np.expm1(2 * s) + 2.0 ** -21) + C * step * (2.0 ** -22 + (max(plan.kv) + 8) * 2.0 ** -24))[:, None, None]


def check_attn(out, ref, bound, what, norm=None):
    """Within the bound everywhere; NaN in ref: a row that the call leaves alone (out holds what it held)."""
    out = np.asarray(out, np.float64)
    live = ~np.isnan(ref)
    err = np.abs(np.where(live, out - ref, 0.0))
    assert np.isfinite(out[live]).all(), what
    worst = float((err / bound).max())
    rel = float(np.linalg.norm(err) / max(np.linalg.norm(np.where(live, ref, 0.0)), 1e-30))
    print(f"  {what}: {worst:.3f} of the bound, {rel:.2e} of the norm", flush=True)
    assert worst <= 1.0, what
    if norm:
        assert rel <= norm, (what, rel)


__all__ = ["TYPES", "NAME", "Plan", "random_cache", "cache_on", "attn_bound", "check_attn", "device", "to_dev"]
