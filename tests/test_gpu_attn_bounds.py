"""mq_attn with bounds below the lengths: rows keep their positions, and keys from max_kv on are left out."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import NAME, TYPES, Plan, attn_bound, bound_for, cache_on, check_attn, device, random_cache, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("kernel", ["attn_few", "attn_many"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 60)])
@pytest.mark.parametrize("max_kv", [1, 50, 64, 600])
def test_lengths_above_max_kv(qtype, kernel, causal, window, max_kv):
    rng = np.random.default_rng([qtype, max_kv, window])
    heads, dim, hq, n, page = 2, 64, 4, 20, 16
    plan = Plan([n, n, 3], [90, 1500, 40], page, rng)
    data = random_cache(qtype, plan, heads, dim, rng)
    q = rng.standard_normal((plan.T, hq, dim)).astype(np.float32)
    dev = device()
    out = mq.attn(cache_on(dev, data, qtype, plan, heads, dim), plan.seqs(dev), to_dev(q, dev), causal=causal, window=window,
                  max_q=bound_for(kernel, plan, hq, heads), max_kv=max_kv).cpu().numpy()
    assert mq.last_kernel() == kernel
    K, V = ko.get(data, qtype, page, heads, dim)
    ref = np.zeros(q.shape)
    for t, (b, pos) in enumerate(ko.rows_of(plan.q_start, plan.kv_len, plan.T)):
        j = np.arange(min(plan.kv[b], max_kv))
        seen = np.ones(len(j), bool)
        if causal:
            seen = (j <= pos) & ((j > pos - window) | (window == 0))
        p, s = plan.table[b, j // page], j % page
        ref[t] = ko.attention(q[t], K[p, :, s].transpose(1, 0, 2), V[p, :, s].transpose(1, 0, 2), seen, dim ** -0.5)
    check_attn(out, ref, attn_bound(data, qtype, plan, heads, dim, q, dim ** -0.5), f"max_kv {max_kv}")
