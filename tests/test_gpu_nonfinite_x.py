"""An infinity or a NaN in x makes every output of mq_gemv_ep NaN, on every kernel and wherever it stands in x; the
next call is not touched by it."""

import pytest

from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import device, say, to_dev, weights
from test_gpu_epilogue import GEMV, laid_out

pytestmark = pytest.mark.gpu

CASES = GEMV + [(mq.Q8_0, 9, 32, "gemv<q8_0>"), (mq.Q8_0, 300, 32768, "gemv<q8_0>"), (mq.Q8_0, 8192, 13 * 256, "gemv_mfma<q8_0>"),
                (mq.Q8_0, 8193, 16 * 256, "gemv_mfma<q8_0>"), (mq.Q5_1, 77, 32768, "gemv<q5_1>")]


@pytest.mark.parametrize("qtype,N,K,kernel", CASES, ids=[f"{g[3]}-{g[1]}x{g[2]}" for g in CASES])
def test_every_output_is_nan(qtype, N, K, kernel):
    import torch
    dev = device()
    say(f"gemv_ep of a non-finite x: {kernel} N={N} K={K}")
    W = laid_out(weights(qtype & 0xFF, N, K, "quantized", 700), qtype, N, K, dev)
    x = to_dev(synth.activations(1, K, config_index=14, tensor_index=7)[0], dev)
    res = torch.ones(N, device=dev)
    clean = mq.gemv_ep(W, qtype, x, N, K, residual=res)
    assert mq.last_kernel() == kernel, mq.last_kernel()
    assert bool(torch.isfinite(clean).all())
    for at in sorted({0, 5, 31, K // 4 + 3, K // 2, 3 * K // 4 - 1, K - 32, K - 1}):
        for value in (float("nan"), float("inf"), -float("inf")):
            bad = x.clone()
            bad[at % K] = value
            for act in (mq.ACT_NONE, mq.ACT_RELU):
                y = mq.gemv_ep(W, qtype, bad, N, K, act=act, residual=res)
                assert bool(torch.isnan(y).all()), (at, value, act, int(torch.isnan(y).sum()))
    big = x * (1e30 / float(x.abs().max()))      # large, but finite: no NaN out of the check itself
    assert bool(torch.isfinite(mq.gemv_ep(W, qtype, big, N, K)).all())
    assert torch.equal(mq.gemv_ep(W, qtype, x, N, K, residual=res), clean)
