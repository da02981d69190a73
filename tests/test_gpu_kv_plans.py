"""Arrays of sequences that describe no valid call: the calls on a paged cache return, and touch nothing but their own tensors."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from gpu_cases import say
from kv_cases import Plan, bound_for, cache_on, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

HQ, HEADS, DIM, PAGE, T = 4, 2, 64, 16, 6
INT_MIN, INT_MAX = -(1 << 31), (1 << 31) - 1


def guarded(a, dev, fill):
    """The array on the device between 256 KiB of `fill` on either side: (its view, a check that the rest is as it was)."""
    import torch
    a = np.ascontiguousarray(a)
    pad = (1 << 18) // a.itemsize
    whole = torch.full((2 * pad + a.size,), fill, dtype=torch.from_numpy(a).dtype, device=dev)
    view = whole[pad:pad + a.size]
    view.copy_(torch.from_numpy(a.reshape(-1)))

    def untouched():
        return bool((whole[:pad] == fill).all()) and bool((whole[pad + a.size:] == fill).all())

    return view.view(*a.shape), untouched


PLANS = {
    "falling starts": ([0, 5, 2, 4], [20, 20, 20]),
    "falling at once": ([6, 4, 2, 0], [20, 20, 20]),
    "starts below zero": ([-3, -1, 2, 6], [20, 20, 20]),
    "starts past the rows": ([0, 2, 40, 900], [20, 20, 20]),
    "first start not zero": ([2, 3, 4, 6], [20, 20, 20]),
    "starts at the ends of int32": ([INT_MIN, INT_MAX, INT_MIN, 6], [20, 20, 20]),
    "lengths at the ends of int32": ([0, 2, 4, 6], [INT_MAX, INT_MIN, -1]),
    "no lengths": ([0, 2, 4, 6], [0, -5, 1]),
}


class Call:
    """A call's arrays and cache, each between guards; what stands behind the table names a page that no table has."""

    def __init__(self, name, seed):
        self.dev = device()
        rng = np.random.default_rng(seed)
        self.q_start, self.kv_len = PLANS[name]
        self.plan = Plan([2, 2, 2], [20, 20, 20], PAGE, rng)
        self.spare = [p for p in range(self.plan.pages) if p not in self.plan.table][0]
        self.checks = []
        starts, lengths = self.guard(np.array(self.q_start, np.int32), 3), self.guard(np.array(self.kv_len, np.int32), 20)
        self.table = self.guard(self.plan.table, self.spare)
        self.data = self.guard(random_cache(mq.Q4_0, self.plan, HEADS, DIM, rng), 171)
        self.cache = mq.KVCache(self.data, mq.Q4_0, self.plan.pages, PAGE, HEADS, DIM)
        self.seqs = mq.KVSeqs(starts, lengths, self.table)
        self.x = to_dev(rng.standard_normal((T, HQ + 2 * HEADS, DIM)).astype(np.float32), self.dev)

    def guard(self, a, fill):
        view, untouched = guarded(a, self.dev, fill)
        self.checks.append(untouched)
        return view

    def rows(self, heads):
        return self.guard(np.full((T, heads, DIM), 777.0, np.float32), 777.0)

    def check(self):
        assert all(c() for c in self.checks)
        assert np.array_equal(self.table.cpu().numpy(), self.plan.table)
        assert self.seqs.kv_len.tolist() == self.kv_len and self.seqs.q_start.tolist() == self.q_start


@pytest.mark.parametrize("name", PLANS)
def test_append_and_read(name):
    import torch
    c = Call(name, 21)
    q_out, kr, vr = c.rows(HQ), c.rows(HEADS), c.rows(HEADS)
    freq = to_dev((10000.0 ** (-np.arange(0, DIM, 2) / DIM)).astype(np.float32), c.dev)
    chunk = HEADS * ko.chunk_bytes(mq.Q4_0, PAGE, DIM)
    spare = slice(c.spare * chunk, (c.spare + 1) * chunk)
    before = c.data[spare].clone()
    say(f"append: {name}")
    mq.kv_append(c.cache, c.seqs, c.x[:, HQ:HQ + HEADS], c.x[:, HQ + HEADS:], q=c.x[:, :HQ], inv_freq=freq, q_out=q_out)
    torch.cuda.synchronize()
    say(f"read: {name}")
    mq.kv_read(c.cache, c.seqs, T, k=kr, v=vr)
    torch.cuda.synchronize()
    c.check()
    assert torch.equal(before, c.data[spare])
    if name == "falling starts":        # rows 0 and 1 are the first sequence's; row 4 is none's
        assert (q_out[0] != 777.0).any() and (q_out[4] == 777.0).all() and (kr[4] == 777.0).all()


@pytest.mark.parametrize("name", PLANS)
@pytest.mark.parametrize("window", [0, 3])
@pytest.mark.parametrize("kernel", ["attn_few", "attn_many"])
def test_attention(name, window, kernel):
    import torch
    c = Call(name, 23)
    q, out = c.guard(c.x[:, :HQ].cpu().numpy(), 0.5), c.rows(HQ)
    say(f"{kernel}: {name}, window {window}")
    mq.attn(c.cache, c.seqs, q, window=window, max_q=bound_for(kernel, c.plan, HQ, HEADS), max_kv=40, out=out)
    torch.cuda.synchronize()
    assert mq.last_kernel() == kernel
    c.check()


def test_a_valid_plan_beside_them():
    """The guard's own arrays with a valid plan: every row is served."""
    import torch
    dev = device()
    rng = np.random.default_rng(22)
    plan = Plan([2, 2, 2], [20, 20, 20], PAGE, rng)
    data = random_cache(mq.Q4_0, plan, HEADS, DIM, rng)
    q = rng.standard_normal((T, HQ, DIM)).astype(np.float32)
    table, c = guarded(plan.table, dev, 1)
    seqs = mq.KVSeqs(to_dev(plan.q_start, dev), to_dev(plan.kv_len, dev), table)
    one = mq.attn(cache_on(dev, data, mq.Q4_0, plan, HEADS, DIM), seqs, to_dev(q, dev), max_q=2, max_kv=20)
    two = mq.attn(cache_on(dev, data, mq.Q4_0, plan, HEADS, DIM), plan.seqs(dev), to_dev(q, dev), max_q=2, max_kv=20)
    assert torch.equal(one, two) and c()
