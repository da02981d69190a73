"""The operators together, as a decoder runs them: q, k and v products of block-quantized weights, norm, rotation and
append, attention over the cache, the output product on the residual stream, the vocabulary head and sampling; a
prompt first, then token by token, against the same in f64 from the weights' and the cache's values."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, device, to_dev

pytestmark = pytest.mark.gpu

HQ, HEADS, DIM, PAGE, VOCAB, EPS = 8, 2, 64, 16, 1000, 1e-6
WIDTH = 512


class Layer:
    def __init__(self, qtype, seed):
        import torch
        rng = np.random.default_rng(seed)
        self.dev, self.qtype = device(), qtype
        make = lambda t, rows, cols: synth.random_blocks(t, rows, cols, rng, exp_lo=-12, exp_hi=-9)   # noqa: E731
        self.raw = dict(qkv=(make(mq.Q4_K, (HQ + 2 * HEADS) * DIM, WIDTH), mq.Q4_K, (HQ + 2 * HEADS) * DIM, WIDTH),
                        out=(make(mq.Q6_K, WIDTH, HQ * DIM), mq.Q6_K, WIDTH, HQ * DIM),
                        head=(make(mq.Q8_0, VOCAB, WIDTH), mq.Q8_0, VOCAB, WIDTH))
        self.W = {k: to_dev(v[0].reshape(-1), self.dev) for k, v in self.raw.items()}
        self.norms = [(1 + 0.1 * rng.standard_normal(DIM)).astype(np.float32) for _ in range(2)]
        self.freq = (10000.0 ** (-np.arange(0, DIM, 2) / DIM)).astype(np.float32)
        self.pages = 12
        self.table = rng.permutation(self.pages).astype(np.int32).reshape(2, 6)
        size = mq.kv_cache_bytes(qtype, self.pages, PAGE, HEADS, DIM)
        self.cache = mq.KVCache(torch.zeros(size, dtype=torch.uint8, device=self.dev), qtype, self.pages, PAGE, HEADS, DIM)
        self.d = {k: to_dev(v, self.dev) for k, v in dict(nq=self.norms[0], nk=self.norms[1], f=self.freq, table=self.table).items()}

    def seqs(self, n, kv):
        i32 = lambda a: to_dev(np.array(a, np.int32), self.dev)   # noqa: E731
        return mq.KVSeqs(i32(np.concatenate([[0], np.cumsum(n)])), i32(kv), self.d["table"])

    def product(self, name, x, residual=None):
        import torch
        _, t, N, K = self.raw[name]
        M = x.shape[0]
        if M > 4:
            return mq.gemm_ep(self.W[name], t, mq.quantize_act(x), M, N, K, residual=residual)
        rows = [mq.gemv_ep(self.W[name], t, x[m], N, K, residual=None if residual is None else residual[m].contiguous()) for m in range(M)]
        return torch.stack(rows)

    def run(self, x, n, kv, u):
        """(residual stream, ids, probabilities, the rotated queries) of rows x."""
        seqs = self.seqs(n, kv)
        qkv = self.product("qkv", x).view(-1, HQ + 2 * HEADS, DIM)
        q = mq.kv_append(self.cache, seqs, qkv[:, HQ:HQ + HEADS], qkv[:, HQ + HEADS:], q=qkv[:, :HQ], q_norm=self.d["nq"],
                         k_norm=self.d["nk"], eps=EPS, inv_freq=self.d["f"])
        o = mq.attn(self.cache, seqs, q, max_q=max(n), max_kv=max(kv))
        y = self.product("out", o.view(-1, HQ * DIM), residual=x)
        logits = self.product("head", y)
        ids, probs = mq.sample(logits, u, top_k=None, top_p=None)
        return qkv, q, o, y, logits, ids, probs


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
def test_a_prompt_and_then_tokens(qtype):
    import torch
    L = Layer(qtype, 60 + qtype)
    rng = np.random.default_rng(qtype)
    w = {k: oracle.decode(v[0], *v[1:]) for k, v in L.raw.items()}
    kv = [0, 0]
    for n in ([37, 20], [1, 1], [1, 1], [2, 1], [1, 0], [9, 5]):
        kv = [a + b for a, b in zip(kv, n)]
        T = sum(n)
        x = rng.standard_normal((T, WIDTH)).astype(np.float32)
        u = rng.random(T).astype(np.float32)
        before = L.cache.data.cpu().numpy()
        got = [t.cpu().numpy() for t in L.run(to_dev(x, L.dev), n, kv, to_dev(u, L.dev))]
        torch.cuda.synchronize()
        qkv, q, o, y, logits, ids, probs = got
        # each operator against f64 from what it was given, so that a difference is its own
        q_start = np.concatenate([[0], np.cumsum(n)])
        at = [p for _, p in ko.rows_of(q_start, kv, T)]
        qr = ko.rotated(ko.normed(qkv[:, :HQ], L.norms[0], EPS), at, L.freq, 1)
        assert np.abs(q - qr).max() <= 2.0 ** -24 * np.abs(qr).max() * 1.0001
        kr = ko.rotated(ko.normed(qkv[:, HQ:HQ + HEADS], L.norms[1], EPS), at, L.freq, 1).astype(np.float32)
        for t, (b, p) in enumerate(ko.rows_of(q_start, kv, T)):
            page, slot = ko.place(L.table, L.pages, PAGE, b, p)
            for h in range(HEADS):
                for which, v in ((0, kr[t, h]), (1, qkv[t, HQ + HEADS + h])):
                    ko.put(before, qtype, PAGE, HEADS, DIM, page, slot, h, which, *ko.quantize(v, qtype))
        assert np.array_equal(before, L.cache.data.cpu().numpy())
        ref = ko.attn(before, qtype, L.pages, PAGE, HEADS, DIM, q_start, kv, L.table, q, DIM ** -0.5)
        assert np.linalg.norm(o - ref) <= 1.5e-6 * np.linalg.norm(ref)
        # the products within their 2e-4 of the row norms (8-bit activations in the many-row form)
        a = o.reshape(T, -1).astype(np.float64)
        bound = np.linalg.norm(a, axis=1)[:, None] * np.linalg.norm(w["out"], axis=1)
        assert np.abs(y - (x + a @ w["out"].T)).max() <= ((2e-4 if T <= 4 else 2e-2) * bound).max()
        for m in range(T):
            assert (ids[m], ) == (ko.sample(logits[m], float(u[m]))[0],)
            assert abs(probs[m] - ko.sample(logits[m], float(u[m]))[1]) <= 2.0 ** -23 * probs[m]
