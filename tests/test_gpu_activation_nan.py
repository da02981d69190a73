"""A NaN is never swallowed by an activation: in a term of the products' epilogues (zero activations make the
product exactly 0, so the bias alone is what the activation gets) and in an expert's gate."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import device, say, to_dev, weights

pytestmark = pytest.mark.gpu

ACTS = {mq.ACT_NONE: "none", mq.ACT_SILU: "silu", mq.ACT_GELU_TANH: "gelu_tanh", mq.ACT_GELU_ERF: "gelu_erf",
        mq.ACT_RELU: "relu"}

PRODUCTS = [  # (type, M, K, kernel): the kernels' ways to store
    (mq.Q8_0, 1, 32, "gemv<q8_0>"), (mq.Q4_K, 1, 3584, "gemv_mfma<q4_K>"), (mq.Q5_0, 3, 64, "gemv_q8<q5_0>"),
    (mq.Q5_1, 40, 64, "mmq<q5_1>"), (mq.Q4_K, 40, 256, "mmq_kw<q4_K>"), (mq.Q4_K | mq.REPACKED, 40, 256, "mmq_f6<q4_K plane>"),
]
IDS = [p[3] for p in PRODUCTS]


class Product:
    """act(0 + bias) through a product of zero activations: run(bias, act) gives [M, N] on the device."""

    def __init__(self, qtype, M, N, K):
        import torch
        self.qtype, self.M, self.N, self.K = qtype, M, N, K
        self.dev = device()
        base = qtype & 0xFF
        W = to_dev(weights(base, N, K, "random", 740).reshape(-1), self.dev)
        self.W = mq.repack(W, base, N, K) if qtype & mq.REPACKED else W
        X = torch.zeros((M, K), device=self.dev)
        self.x = X[0].contiguous() if M == 1 else mq.quantize_act(X)

    def run(self, bias, act, **terms):
        if self.M == 1:
            return mq.gemv_ep(self.W, self.qtype, self.x, self.N, self.K, bias=bias, act=act, **terms).view(1, self.N)
        return mq.gemm_ep(self.W, self.qtype, self.x, self.M, self.N, self.K, bias=bias, act=act, **terms)


@pytest.mark.parametrize("act", ACTS, ids=ACTS.values())
@pytest.mark.parametrize("qtype,M,K,kernel", PRODUCTS, ids=IDS)
def test_a_nan_stays(qtype, M, K, kernel, act):
    import torch
    N = 8224 if M == 1 else 1000
    p = Product(qtype, M, N, K)
    rng = np.random.default_rng(8)
    bias = rng.standard_normal(N).astype(np.float32)
    res = to_dev(rng.standard_normal((M, N)).astype(np.float32), p.dev)
    say(f"{kernel} {ACTS[act]}: a NaN in the bias")
    at = [0, 17, N // 2, N - 1]
    keep = np.setdiff1d(np.arange(N), at)
    for terms in ({}, dict(mul=res, residual=res)):
        clean = p.run(to_dev(bias, p.dev), act, **terms).cpu().numpy()
        bad = bias.copy()
        bad[at] = np.nan
        y = p.run(to_dev(bad, p.dev), act, **terms).cpu().numpy()
        assert mq.last_kernel() == kernel, mq.last_kernel()
        assert np.all(np.isnan(y[:, at])), y[:, at]
        assert np.array_equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("act", ACTS, ids=ACTS.values())
@pytest.mark.parametrize("M", [1, 5])
def test_a_nan_gate_reaches_the_token(M, act):
    """A gate row whose weights are NaN while the up row is finite: by the formula every output of the tokens
    that chose the expert is NaN."""
    import torch
    E, F, K = 4, 256, 256
    dev = device()
    rng = np.random.default_rng(9)
    g, u = (synth.random_blocks(mq.Q8_0, E * F, K, rng, exp_lo=-12, exp_hi=-8).reshape(E * F, -1) for _ in range(2))
    d = synth.random_blocks(mq.Q4_K, E * K, F, rng, exp_lo=-12, exp_hi=-8)
    X = to_dev(rng.standard_normal((M, K)).astype(np.float32), dev)
    ids = np.tile(np.array([0, 1], np.int32), (M, 1))
    ids[0] = [1, 2]                                  # token 0 chooses the expert below, the others do not
    wts = to_dev(np.full((M, 2), 0.5, np.float32), dev)
    ids[1:, 1] = 3
    say(f"moe M={M} {ACTS[act]}: a NaN in the gate")

    def run(gate):
        Y = mq.moe_ffn(to_dev(gate.reshape(-1), dev), to_dev(u.reshape(-1), dev), mq.Q8_0, to_dev(d.reshape(-1), dev), mq.Q4_K,
                       X, to_dev(ids, dev), wts, E, F, act=act)
        torch.cuda.synchronize()
        return Y.cpu().numpy()

    clean = run(g)
    assert np.all(np.isfinite(clean))
    bad = g.copy()
    bad[2 * F + 7, 0:2] = (0x00, 0x7E)               # expert 2, row 7: the first block's scale is NaN
    y = run(bad)
    assert np.all(np.isnan(y[0]))
    assert np.array_equal(y[1:], clean[1:])
