"""The output of mq_gemv_ep and mq_gemm_ep may be the multiplier, the residual, or both: on every kernel, with the
bits of the same call into memory of its own."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq, synth

from gpu_cases import device, say, to_dev, weights
from test_gpu_epilogue import FILLED, GEMM, GEMV, laid_out

pytestmark = pytest.mark.gpu


def in_place(call, M, N, dev, what):
    """call(out, **terms) -> out."""
    import torch
    rng = np.random.default_rng(31)
    mul, res = (to_dev(rng.standard_normal((M, N)).astype(np.float32), dev) for _ in range(2))
    bias = to_dev(rng.standard_normal(N).astype(np.float32), dev)
    for act in (mq.ACT_NONE, mq.ACT_SILU):
        for give in (("mul",), ("residual",), ("mul", "residual")):
            terms = {k: v for k, v in (("mul", mul), ("residual", res)) if k in give}
            want = call(torch.full((M, N), float("nan"), device=dev), bias=bias, act=act, **terms)
            for name in give:
                mine = {k: v.clone() for k, v in terms.items()}
                call(mine[name], bias=bias, act=act, **mine)
                assert torch.equal(mine[name], want), f"{what}: into {name} of {give}, act {act}"
                for k, v in terms.items():
                    assert k == name or torch.equal(mine[k], v)
    both = mul.clone()
    call(both, bias=None, act=mq.ACT_NONE, mul=both, residual=both)
    assert torch.equal(both, call(torch.empty_like(mul), bias=None, act=mq.ACT_NONE, mul=mul, residual=mul)), what


@pytest.mark.parametrize("qtype,N,K,kernel", GEMV, ids=[f"{g[3]}-{g[1]}x{g[2]}" for g in GEMV])
def test_gemv(qtype, N, K, kernel):
    dev = device()
    say(f"gemv_ep in place {kernel} N={N} K={K}")
    W = laid_out(weights(qtype & 0xFF, N, K, "quantized", 700), qtype, N, K, dev)
    x = to_dev(synth.activations(1, K, config_index=14, tensor_index=7)[0], dev)
    in_place(lambda y, **t: mq.gemv_ep(W, qtype, x, N, K, y=y, **t), 1, N, dev, kernel)
    assert mq.last_kernel() == kernel


CASES = [g[:5] for g in GEMM] + [(t, M, N, K, f"own split of {rows} rows") for t, M, N, K, rows in FILLED]


@pytest.mark.parametrize("qtype,M,N,K,kernel", CASES, ids=[f"{g[4]}-{g[0]}-{g[1]}x{g[2]}x{g[3]}" for g in CASES])
def test_gemm(qtype, M, N, K, kernel):
    import torch
    dev = device()
    say(f"gemm_ep in place {kernel} M={M} N={N} K={K}")
    W = laid_out(weights(qtype & 0xFF, N, K, "quantized", 710), qtype, N, K, dev)
    Xq = mq.quantize_act(to_dev(synth.activations(M, K, config_index=14, tensor_index=8), dev))
    size = (mq.gemm_ep_scratch_bytes if kernel.startswith("own") else mq.gemm_scratch_bytes)(qtype, M, N, K)
    scratch = torch.zeros(max(16, size), dtype=torch.uint8, device=dev)
    in_place(lambda Y, **t: mq.gemm_ep(W, qtype, Xq, M, N, K, Y=Y, scratch=scratch, **t), M, N, dev, kernel)
    assert kernel.startswith("own") or mq.last_kernel() == kernel
