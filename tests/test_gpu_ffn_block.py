"""The feed-forward operators together, as a decoder layer runs them, against the oracle in f64:
router, experts and a shared dense expert added to the residual stream; eagerly, on another stream
than the current one, and captured into graphs that are replayed with other inputs between."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import device, say, to_dev

pytestmark = pytest.mark.gpu

E, K, F, FS, TOPK = 16, 512, 256, 768, 4    # experts, width, expert and shared-expert hidden sizes


class Block:
    def __init__(self, M, dense_gemm):
        import torch
        rng = np.random.default_rng(40 + M)
        make = lambda t, rows, cols: synth.random_blocks(t, rows, cols, rng, exp_lo=-12, exp_hi=-8)   # noqa: E731
        self.M, self.dense_gemm = M, dense_gemm
        self.raw = dict(g=make(mq.Q4_K, E * F, K), u=make(mq.Q4_K, E * F, K), d=make(mq.Q6_K, E * K, F),
                        sg=make(mq.Q8_0, FS, K), su=make(mq.Q8_0, FS, K), sd=make(mq.Q6_K, K, FS))
        self.Wr = (rng.standard_normal((E, K)) * 0.1).astype(np.float32)
        self.dev = device()
        self.W = {k: to_dev(v.reshape(-1), self.dev) for k, v in self.raw.items()}
        self.Wrd = to_dev(self.Wr, self.dev)
        self.route_scratch = torch.zeros(mq.moe_route_scratch_bytes(M, K, E), dtype=torch.uint8, device=self.dev)
        self.moe_scratch = torch.zeros(mq.moe_scratch_bytes(M, TOPK, F, K), dtype=torch.uint8, device=self.dev)
        need = max(mq.gemm_scratch_bytes(mq.Q8_0, M, FS, K), mq.gemm_scratch_bytes(mq.Q6_K, M, K, FS), 16)
        self.gemm_scratch = torch.zeros(need, dtype=torch.uint8, device=self.dev)

    def run(self, X, Y):
        """Y = X + experts(X) + shared(X); every call on the current stream."""
        W, M = self.W, self.M
        ids, wts = mq.moe_route(X, self.Wrd, TOPK, scratch=self.route_scratch)
        mq.moe_ffn(W["g"], W["u"], mq.Q4_K, W["d"], mq.Q6_K, X, ids, wts, E, F, residual=X, Y=Y,
                   scratch=self.moe_scratch)
        if self.dense_gemm:
            Xq = mq.quantize_act(X)
            u = mq.gemm_ep(W["su"], mq.Q8_0, Xq, M, FS, K, scratch=self.gemm_scratch)
            h = mq.gemm_ep(W["sg"], mq.Q8_0, Xq, M, FS, K, act=mq.ACT_SILU, mul=u, scratch=self.gemm_scratch)
            mq.gemm_ep(W["sd"], mq.Q6_K, mq.quantize_act(h), M, K, FS, residual=Y, Y=Y, scratch=self.gemm_scratch)
        else:
            for m in range(M):
                x, y = X[m], Y[m]
                u = mq.gemv(W["su"], mq.Q8_0, x, FS, K)
                h = mq.gemv_ep(W["sg"], mq.Q8_0, x, FS, K, act=mq.ACT_SILU, mul=u, y=u)
                mq.gemv_ep(W["sd"], mq.Q6_K, h, K, FS, residual=y, y=y)
        return ids

    def oracle(self, X):
        ids, wts = oracle.moe_route(X, self.Wr, TOPK)
        Y, _ = oracle.moe_ffn(self.raw["g"], self.raw["u"], mq.Q4_K, self.raw["d"], mq.Q6_K, X, ids, wts, E, F, 1, X)
        w = {k: oracle.decode(self.raw[k], t, *s) for k, t, s in (("sg", mq.Q8_0, (FS, K)), ("su", mq.Q8_0, (FS, K)),
                                                                  ("sd", mq.Q6_K, (K, FS)))}
        x = X.astype(np.float64)
        Y = Y + (oracle.activation(x @ w["sg"].T, 1) * (x @ w["su"].T)) @ w["sd"].T
        return Y, ids

    def check(self, X, Y, what):
        ref, _ = self.oracle(X)
        rel = np.linalg.norm(Y - ref, axis=1) / np.linalg.norm(ref, axis=1)
        say(f"ffn block M={self.M} {what}: relative {rel.max():.2e}")
        # f32 decode: the products' accuracy; the prefill products take 8-bit activations twice (an error of
        # 1 / 254 of each block's maximum at most: a few times 1/254 / sqrt(3) of the norm for normal values)
        assert rel.max() <= (3e-2 if self.dense_gemm else 1e-5), what


def inputs(M, seed):
    return np.random.default_rng(seed).standard_normal((M, K)).astype(np.float32)


@pytest.mark.parametrize("M,dense_gemm", [(1, False), (3, False), (40, True)])
def test_eager(M, dense_gemm):
    import torch
    b = Block(M, dense_gemm)
    X = inputs(M, 1)
    Xd, Y = to_dev(X, b.dev), torch.empty((M, K), device=b.dev)
    ids = b.run(Xd, Y)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), b.oracle(X)[1])
    b.check(X, Y.cpu().numpy(), "eager")


@pytest.mark.parametrize("M,dense_gemm", [(1, False), (40, True)])
def test_side_stream(M, dense_gemm):
    import torch
    b = Block(M, dense_gemm)
    X = inputs(M, 2)
    Xd, Y, Y2 = to_dev(X, b.dev), torch.empty((M, K), device=b.dev), torch.empty((M, K), device=b.dev)
    b.run(Xd, Y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.run(Xd, Y2)
    s.synchronize()
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("M,dense_gemm", [(1, False), (3, False), (40, True)])
def test_two_captured_graphs_share_the_workspaces(M, dense_gemm):
    """Two graphs of the block over the same scratch buffers, replayed in turn with eager calls and
    new inputs between: every replay gives the eager bits."""
    import torch
    b = Block(M, dense_gemm)
    Xa, Xb = torch.empty((M, K), device=b.dev), torch.empty((M, K), device=b.dev)
    Ya, Yb, Ye = (torch.empty((M, K), device=b.dev) for _ in range(3))
    Xa.copy_(to_dev(inputs(M, 3), b.dev))
    Xb.copy_(to_dev(inputs(M, 4), b.dev))
    b.run(Xa, Ye)
    torch.cuda.synchronize()
    graphs = []
    for X, Y in ((Xa, Ya), (Xb, Yb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run(X, Y)
        graphs.append(g)
    for turn in range(4):
        say(f"ffn block graphs M={M} replay {turn}")
        for X, Y, g in ((Xa, Ya, graphs[0]), (Xb, Yb, graphs[1])):
            X.copy_(to_dev(inputs(M, 10 * turn + (X is Xb)), b.dev))
            Y.fill_(float("nan"))
            g.replay()
            b.run(X, Ye)
            torch.cuda.synchronize()
            assert torch.equal(Y, Ye), turn
