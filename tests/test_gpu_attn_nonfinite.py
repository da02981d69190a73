"""mq_attn over contexts that are cut into pieces, with what is not finite in queries, keys and values: NaN where it is used,
the clean call's bits everywhere else."""

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

from gpu_cases import say
from kv_cases import NAME, TYPES, Plan, bound_for, cache_on, device, random_cache, to_dev

pytestmark = pytest.mark.gpu

KERNELS = ["attn_few", "attn_many"]
HQ, HEADS, DIM, PAGE = 6, 2, 64, 32
# of these lengths the first two leave the newest token alone in a piece of attn_few (pieces of nine steps of 32 keys)
LENGTHS = [2881, 2593, 2700, 40]


class Case:
    def __init__(self, qtype, kernel, n, seed):
        rng = np.random.default_rng([qtype, n, seed])
        self.qtype, self.kernel = qtype, kernel
        self.plan = Plan([n] * len(LENGTHS), LENGTHS, PAGE, rng)
        self.data = random_cache(qtype, self.plan, HEADS, DIM, rng)
        self.q = rng.standard_normal((self.plan.T, HQ, DIM)).astype(np.float32)
        self.max_q = bound_for(kernel, self.plan, HQ, HEADS)
        # pieces are joined
        assert mq.attn_scratch_bytes(qtype, len(LENGTHS), HQ, HEADS, DIM, self.max_q, self.plan.max_kv) > 1 << 18
        self.clean = self.call(self.data, self.q)
        assert np.isfinite(self.clean).all()

    def call(self, data, q, **kw):
        dev = device()
        out = mq.attn(cache_on(dev, data, self.qtype, self.plan, HEADS, DIM), self.plan.seqs(dev), to_dev(q, dev), max_q=self.max_q,
                      max_kv=self.plan.max_kv, **kw)
        assert mq.last_kernel() == self.kernel
        return out.cpu().numpy()

    def with_scale(self, which, b, pos, head, dim, value):
        """The cache with another scale of one block of a key (which 4) or a value (5)."""
        raw = self.data.copy().reshape(self.plan.pages, HEADS, -1)
        page, slot = ko.place(self.plan.table, self.plan.pages, PAGE, b, pos)
        s = ko.places(self.qtype, PAGE, DIM)[which][slot, dim]
        raw[page, head, s:s + 2] = np.frombuffer(np.float16(value).tobytes(), np.uint8)
        return raw.reshape(-1)

    def row(self, b, i):
        return int(self.plan.q_start[b]) + i


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_bad_query(n, bad, kernel):
    c = Case(mq.Q4_0, kernel, n, 1)
    for b in range(len(LENGTHS)):
        say(f"sequence {b}")
        q = c.q.copy()
        q[c.row(b, n - 1), 4, 17] = bad
        want = c.clean.copy()
        want[c.row(b, n - 1), 4] = np.nan
        assert np.array_equal(c.call(c.data, q), want, equal_nan=True)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("kernel", KERNELS)
def test_a_nan_key_or_value(qtype, n, kernel):
    """The newest token (in two of the sequences the only key of a piece), one amid a piece, and the first one."""
    c = Case(qtype, kernel, n, 2)
    for b, l in enumerate(LENGTHS):
        for pos in (l - 1, l // 2, 0):
            for which in (4, 5):
                say(f"sequence {b}, position {pos}, {'key' if which == 4 else 'value'}")
                got = c.call(c.with_scale(which, b, pos, 1, 33, np.nan), c.q)
                want = c.clean.copy()
                for i in range(n):
                    if l - n + i >= pos:
                        want[c.row(b, i), 3:, 0 if which == 4 else 32:] = np.nan
                assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("kernel", KERNELS)
def test_nothing_but_nan_keys(kernel):
    """Every key of a sequence: every piece's scores are NaN."""
    c = Case(mq.Q4_0, kernel, 2, 3)
    raw = c.data.copy().reshape(c.plan.pages, HEADS, -1)
    nan = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)
    for pos in range(LENGTHS[1]):
        page, slot = ko.place(c.plan.table, c.plan.pages, PAGE, 1, pos)
        s = ko.places(c.qtype, PAGE, DIM)[4][slot, 0]
        raw[page, 0, s:s + 2] = nan
    want = c.clean.copy()
    want[c.row(1, 0):c.row(1, 2), :3] = np.nan
    assert np.array_equal(c.call(raw.reshape(-1), c.q), want, equal_nan=True)


@pytest.mark.parametrize("qtype", TYPES, ids=NAME.get)
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("bad", [np.inf, -np.inf])
@pytest.mark.parametrize("kernel", KERNELS)
def test_an_infinite_key_or_value(qtype, n, bad, kernel):
    """A block whose scale is an infinity (no append makes one; a cache may be filled otherwise): codes of both signs times it are
    infinities of both signs, whatever the sign of the score that they would give."""
    c = Case(qtype, kernel, n, 4)
    for b, l in enumerate(LENGTHS):
        for pos in (l - 1, l // 2, 0):
            for which in (4, 5):
                say(f"sequence {b}, position {pos}, {'key' if which == 4 else 'value'}")
                got = c.call(c.with_scale(which, b, pos, 1, 33, bad), c.q)
                want = c.clean.copy()
                for i in range(n):
                    if l - n + i >= pos:
                        want[c.row(b, i), 3:, 0 if which == 4 else 32:] = np.nan
                assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("window", [8, 40])
@pytest.mark.parametrize("kernel", KERNELS)
def test_infinite_keys_out_of_sight(window, kernel):
    """Infinite scales just outside a window and behind a row's own position."""
    c = Case(mq.Q4_0, kernel, 2, 5)
    raw = c.data.copy().reshape(c.plan.pages, HEADS, -1)
    inf = np.frombuffer(np.float16(-np.inf).tobytes(), np.uint8)
    clean = c.call(c.data, c.q, window=window)
    for b, l in enumerate(LENGTHS):
        if l - 2 - window < 0:       # the window covers the sequence
            continue
        page, slot = ko.place(c.plan.table, c.plan.pages, PAGE, b, l - 2 - window)      # the first row's first key is one further
        for which in (4, 5):
            for s in np.unique(ko.places(c.qtype, PAGE, DIM)[which][slot]):
                raw[page, :, s:s + 2] = inf
    assert np.array_equal(c.call(raw.reshape(-1), c.q, window=window), clean)
