"""How the calls on a paged cache and mq_sample run rather than what they compute: refused launches, streams,
two calls at once, captured graphs and the workspaces they leave behind."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from gpu_cases import say
from kv_cases import Plan, attn_bound, cache_on, check_attn, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

NAMES = ("kv_append", "kv_read", "attn", "attn_many", "sample", "sample_row")


class Calls:
    """Each call with inputs of its own on the device; run(name, **kw) gives its outputs."""

    def __init__(self, seed=0):
        dev = device()
        rng = np.random.default_rng(700 + seed)
        normal = lambda *s: to_dev(rng.standard_normal(s).astype(np.float32), dev)   # noqa: E731
        self.dev, self.heads, self.dim, self.hq = dev, 2, 64, 6
        self.plan = Plan([1, 1, 2], [900, 5, 1300], 32, rng)
        self.data = random_cache(mq.Q4_0, self.plan, self.heads, self.dim, rng)
        self.cache, self.seqs = cache_on(dev, self.data, mq.Q4_0, self.plan, self.heads, self.dim), self.plan.seqs(dev)
        self.q, self.k, self.v = normal(4, self.hq, self.dim), normal(4, self.heads, self.dim), normal(4, self.heads, self.dim)
        self.freq = to_dev((10000.0 ** (-np.arange(0, 64, 2) / 64)).astype(np.float32), dev)
        self.many = Plan([50, 30], [800, 31], 32, rng)
        self.many_data = random_cache(mq.Q4_0, self.many, self.heads, self.dim, rng)
        self.many_cache, self.many_seqs = cache_on(dev, self.many_data, mq.Q4_0, self.many, self.heads, self.dim), self.many.seqs(dev)
        self.many_q = normal(80, self.hq, self.dim)
        self.logits, self.short = 2 * normal(3, 20000), 2 * normal(5, 3000)
        self.u = to_dev(rng.random(5).astype(np.float32), dev)
        self.p, self.top_k = to_dev(np.full(5, 0.8, np.float32), dev), to_dev(np.full(5, 300, np.int32), dev)

    def run(self, name, **kw):
        return getattr(self, name)(**kw)

    def kv_append(self, **kw):
        out = mq.kv_append(self.cache, self.seqs, self.k, self.v, q=self.q, inv_freq=self.freq, **kw)
        return out, self.cache.data

    def kv_read(self, **kw):
        return mq.kv_read(self.cache, self.seqs, 4, **kw)

    def attn(self, **kw):
        return (mq.attn(self.cache, self.seqs, self.q, max_q=2, max_kv=1300, **kw),)

    def attn_many(self, **kw):
        return (mq.attn(self.many_cache, self.many_seqs, self.many_q, max_q=1100, max_kv=800, **kw),)

    def sample(self, **kw):
        return mq.sample(self.logits, self.u[:3], top_p=self.p[:3], top_k=self.top_k[:3], **kw)

    def sample_row(self, **kw):
        return mq.sample(self.short, self.u, top_p=self.p, **kw)

    def scratch(self, name):
        import torch
        size = {"attn": lambda: mq.attn_scratch_bytes(mq.Q4_0, 3, 6, 2, 64, 2, 1300),
                "attn_many": lambda: mq.attn_scratch_bytes(mq.Q4_0, 2, 6, 2, 64, 1100, 800),
                "sample": lambda: mq.sample_scratch_bytes(3, 20000), "sample_row": lambda: mq.sample_scratch_bytes(5, 3000)}
        return torch.zeros(max(size[name](), 16), dtype=torch.uint8, device=self.dev)


CALL = {"attn_many": "attn", "sample_row": "sample"}
COUNTERS = {"attn": 1 << 18, "sample": 4 << 20}


@pytest.mark.parametrize("name", NAMES)
def test_a_refused_launch_is_reported_and_leaves_nothing_behind(name):
    import torch
    lib = mq.load()
    c = Calls()
    say(f"refused launch: {name}")
    before = [t.clone() for t in c.run(name)]
    assert lib.mq_debug_refuse_launches(1) == 0
    with pytest.raises(mq.MQError) as e:
        c.run(name)
    assert e.value.code == -7, e.value
    msg = mq.last_error()
    assert f"mq_{CALL.get(name, name)}: launch of" in msg and "refused" in msg, msg
    for a, b in zip(before, c.run(name)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_other_streams(name):
    """On a side stream, by its handle from the default one, and by handle 0 from the side stream, the other one busy: what the
    binding makes belongs to the stream it is given."""
    import torch
    c = Calls()
    ref = [t.clone() for t in c.run(name)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def busy():
        x = torch.randn(2048, 2048, device=c.dev)
        for _ in range(4):
            x = (x @ x).clamp_(-1, 1)
        junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=c.dev) for _ in range(8)]
        del junk

    for turn in range(4):
        say(f"{name}, turn {turn}")
        with torch.cuda.stream(side):
            out = c.run(name)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out))
        busy()
        out = c.run(name, stream=side.cuda_stream)
        side.synchronize()
        assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(ref, out))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy()
            out = c.run(name, stream=0)
        torch.cuda.default_stream().synchronize()
        assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(ref, out))
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["attn", "attn_many", "sample", "sample_row"])
def test_two_calls_at_once(name):
    """On two streams, a workspace each."""
    import torch
    c, d = Calls(), Calls(seed=1)
    refs = [c.run(name), d.run(name)]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = c.scratch(name), d.scratch(name)
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        with torch.cuda.stream(s):
            x = c.run(name, scratch=a)
        with torch.cuda.stream(t):
            y = d.run(name, scratch=b)
        outs.append((x, y))
    torch.cuda.synchronize()
    for pair in outs:
        for got, ref in zip(pair, refs):
            assert all(torch.equal(g, r) for g, r in zip(got, ref))
    counters = COUNTERS[CALL.get(name, name)]
    assert int(a[:counters].sum()) == 0 == int(b[:counters].sum())


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """A graph of the call, replayed with other inputs between, beside eager calls with the same workspace."""
    import torch
    c, d = Calls(), Calls(seed=2)
    kw = {} if name.startswith("kv") else {"scratch": c.scratch(name)}
    c.run(name, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = c.run(name, **kw)
    torch.cuda.synchronize()
    first = {f: getattr(c, f).clone() for f in ("q", "k", "v", "many_q", "logits", "short", "u")}
    for turn in range(6):
        src = d if turn % 2 else None
        for f, t in first.items():
            getattr(c, f).copy_(t if src is None else getattr(d, f))
        graph.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        eager = c.run(name, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), turn


def test_lengths_change_between_replays():
    """A graph of append and attention made for the largest lengths serves every step: the arrays are read when it runs."""
    import torch
    dev = device()
    rng = np.random.default_rng(5)
    heads, dim, hq, page = 2, 128, 8, 16
    plan = Plan([1, 1], [400, 400], page, rng)
    data = random_cache(mq.Q4_0, plan, heads, dim, rng)
    cache, seqs = cache_on(dev, data, mq.Q4_0, plan, heads, dim), plan.seqs(dev)
    x = to_dev(rng.standard_normal((2, hq + 2 * heads, dim)).astype(np.float32), dev)
    freq = to_dev((10000.0 ** (-np.arange(0, dim, 2) / dim)).astype(np.float32), dev)
    scratch = torch.zeros(mq.attn_scratch_bytes(mq.Q4_0, 2, hq, heads, dim, 1, 400), dtype=torch.uint8, device=dev)

    def step():
        q = mq.kv_append(cache, seqs, x[:, hq:hq + heads], x[:, hq + heads:], q=x[:, :hq], inv_freq=freq)
        return q, mq.attn(cache, seqs, q, max_q=1, max_kv=400, scratch=scratch)

    step()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = step()
    torch.cuda.synchronize()
    for lengths in ([1, 399], [17, 2], [0, 33], [400, 256]):
        x.copy_(to_dev(rng.standard_normal(x.shape).astype(np.float32), dev))
        seqs.kv_len.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        q, o = out[0].cpu().numpy(), out[1].cpu().numpy()
        now = cache.data.cpu().numpy()
        plan.kv_len = np.array(lengths, np.int32)
        ref = ko.attn(now, mq.Q4_0, plan.pages, page, heads, dim, plan.q_start, plan.kv_len, plan.table, q, dim ** -0.5)
        check_attn(o, ref, attn_bound(now, mq.Q4_0, plan, heads, dim, q, dim ** -0.5), f"lengths {lengths}", 1e-6)
        e = step()
        assert torch.equal(e[1], out[1])
