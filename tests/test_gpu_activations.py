"""The activations of the epilogues and of the expert layer, value by value: zero activations make every product
exactly 0, so the bias alone is what the activation gets.

Bounds, in half steps of f32 (2^-24 relative), counted operation by operation:

* none, relu: nothing is computed, the value exactly.
* silu, v * 1 / (1 + e): e = 2^t by the exp2 instruction (one step: 2) times its correction (one rounding: 1;
  what the correction itself leaves out is below 2^-30), 1 + e (1), the reciprocal instruction (one step: 2), the
  product (1): 7, and one for their second order.
* gelu (tanh form), v * logistic(u): as silu, and u is off by at most 6 (0.044715 and its product 2, v * v 1, the fma
  1, 1.5957691 and its product 2), which the logistic function amplifies by |u| (1 - logistic(u)).
* gelu (erf), v / 2 * erfc(-v / sqrt 2): erfc within 16 steps (OpenCL's limit for it: 32), the product 1, and the
  argument's 2 amplified by |t erfc'(t) / erfc(t)|, t = -v / sqrt 2.

The values end where the quotient (or erfc) is no longer a normal number (2^-126); a test of its own looks below."""

import numpy as np
import pytest

import oracle
from block_quantized_matmul_mq_amd import mq

from gpu_cases import say, to_dev
from test_gpu_activation_nan import ACTS, IDS, PRODUCTS, Product

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24
LOWEST = {mq.ACT_NONE: -87.0, mq.ACT_SILU: -87.0, mq.ACT_GELU_TANH: -10.0, mq.ACT_GELU_ERF: -12.5, mq.ACT_RELU: -87.0}


def reference(v, act):
    """(act(v) in f64, with no cancellation at any v; relative bound)."""
    from scipy.special import erfc, erfcx
    v = v.astype(np.float64)
    if act == mq.ACT_SILU:
        return v / (1 + np.exp(-v)), 8 * HALF + 0 * v
    if act == mq.ACT_GELU_TANH:
        u = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        return v / (1 + np.exp(-u)), (8 + 6 * np.abs(u) / (1 + np.exp(np.minimum(u, 700.0)))) * HALF
    if act == mq.ACT_GELU_ERF:
        t = -v / np.sqrt(2)
        slope = np.abs(t) * 2 / np.sqrt(np.pi) / erfcx(np.maximum(t, -5))     # (below -5: e^-25, nothing)
        return 0.5 * v * erfc(t), (34 + 2 * slope) * HALF
    return (np.maximum(v, 0) if act == mq.ACT_RELU else v), 0 * v


def test_the_reference_by_hand():
    for act, v, want in ((mq.ACT_SILU, -80.0, -80 * np.exp(-80.0)), (mq.ACT_GELU_ERF, 1.0, 0.8413447460685429),
                         (mq.ACT_GELU_TANH, 1.0, 0.8411919906082768), (mq.ACT_RELU, -3.0, 0.0), (mq.ACT_NONE, -3.0, -3.0)):
        got = reference(np.array([v], np.float32), act)[0][0]
        assert abs(got - want) <= 1e-12 * abs(want)
        assert abs(oracle.activation(v, act) - got) <= 1e-14


@pytest.mark.parametrize("act", ACTS, ids=ACTS.values())
@pytest.mark.parametrize("qtype,M,K,kernel", PRODUCTS, ids=IDS)
def test_every_value(qtype, M, K, kernel, act):
    import torch
    N = 9001 if M == 1 else 1501
    p = Product(qtype, M, N, K)
    worst = 0.0
    for lo, hi in ((LOWEST[act], 87.0), (-3.0, 3.0), (-1e-3, 1e-3)):
        v = np.linspace(lo, hi, N).astype(np.float32)
        y = p.run(to_dev(v, p.dev), act)
        assert mq.last_kernel() == kernel, mq.last_kernel()
        torch.cuda.synchronize()
        y = y.cpu().numpy().astype(np.float64)
        ref, bound = reference(v, act)
        err = np.abs(y - ref) / np.maximum(np.abs(ref), 2.0 ** -126)
        worst = max(worst, float(err.max() / HALF))
        at = int(np.argmax((err - bound).max(axis=0)))
        assert np.all(err <= bound), f"v={v[at]}: {err[:, at].max() / HALF} half steps, {bound[at] / HALF} allowed"
    say(f"{kernel} {ACTS[act]}: worst {worst:.1f} half steps")


@pytest.mark.parametrize("act", [mq.ACT_SILU, mq.ACT_GELU_TANH, mq.ACT_GELU_ERF], ids=["silu", "gelu_tanh", "gelu_erf"])
def test_where_the_quotient_is_no_normal_number(act):
    """Below LOWEST the result is tiny: off by no more than v times the least normal number, never a NaN."""
    import torch
    N = 4001
    p = Product(mq.Q8_0, 1, N, 32)
    for lo in (-150.0, -1e4, -3e38):
        v = np.linspace(lo, LOWEST[act], N).astype(np.float32)
        y = p.run(to_dev(v, p.dev), act)
        torch.cuda.synchronize()
        with np.errstate(over="ignore", invalid="ignore"):
            ref, bound = reference(v, act)
        err = np.abs(y.cpu().numpy()[0] - ref)
        limit = np.where(np.isfinite(bound), bound, 1.0) * np.abs(ref) + np.abs(v.astype(np.float64)) * 2.0 ** -126
        assert np.all(err <= limit), float(v[np.argmax(err - limit)])
