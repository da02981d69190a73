"""Which kernel serves a call of mq_sample: rows of at most two blocks of 2048 tokens whole, longer ones over workgroups and
launches, whatever the number of rows; the token is the oracle's on both sides of the border."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from kv_cases import device, to_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,kernel", [(1, "sample_row"), (2048, "sample_row"), (2049, "sample_row"), (4096, "sample_row"), (4097, "sample"),
                                      (8192, "sample"), (20481, "sample")])
@pytest.mark.parametrize("M", [1, 255, 256, 257])
def test_kernel_by_length(V, M, kernel):
    rng = np.random.default_rng([V, M])
    dev = device()
    l = (2.5 * rng.standard_normal((M, V))).astype(np.float32)
    u, p = rng.random(M).astype(np.float32), rng.uniform(0.5, 1.0, M).astype(np.float32)
    k = rng.integers(0, 60, M).astype(np.int32)
    ids, _ = mq.sample(to_dev(l, dev), to_dev(u, dev), top_k=to_dev(k, dev), top_p=to_dev(p, dev))
    assert mq.last_kernel() == kernel
    ids = ids.cpu().numpy()
    for m in list(range(0, M, 37)) + [M - 1]:
        assert ids[m] == ko.sample(l[m], float(u[m]), 1.0, int(k[m]), float(p[m]))[0], m
    if V > 1:
        mq.sample(to_dev(l, dev), to_dev(u, dev))
        assert mq.last_kernel() == kernel
