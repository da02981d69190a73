"""CPU checks of the paged cache's operators and of sampling: sizes and refusals before any HIP call, the cache's
layout, and the oracle pinned by values worked by hand."""

import ctypes

import numpy as np
import pytest

from block_quantized_matmul_mq_amd import mq
from oracle import kv_oracle as ko

FAKE = 0x10000
BIG = 1 << 40


def cache(data=FAKE, t=mq.Q4_0, pages=8, page=32, heads=4, dim=128):
    c = mq._Cache(data, t, pages, page, heads, dim)
    return ctypes.addressof(c), c


def seqs(q_start=FAKE, kv_len=FAKE, table=FAKE, B=3, width=4):
    s = mq._Seqs(q_start, kv_len, table, B, width)
    return ctypes.addressof(s), s


def append(c=None, s=None, q=FAKE, qs=1024, k=FAKE, ks=512, v=FAKE, vs=512, out=FAKE, os_=1024, T=5, hq=8, qn=None, kn=None,
           eps=1e-6, rope=1, f=FAKE, rot=128, pos=None):
    a, b = c or cache(), s or seqs()
    return mq.load().mq_kv_append(a and a[0], b and b[0], q, qs, k, ks, v, vs, out, os_, T, hq, qn, kn, eps, rope, f, rot, pos, None)


def read(c=None, s=None, T=5, k=FAKE, v=FAKE):
    a, b = c or cache(), s or seqs()
    return mq.load().mq_kv_read(a[0], b[0], T, k, v, None)


def attn(c=None, s=None, q=FAKE, qs=1024, out=FAKE, T=5, hq=8, scale=0.1, causal=1, window=0, mq_=5, mkv=100, scr=FAKE, sb=BIG):
    a, b = c or cache(), s or seqs()
    return mq.load().mq_attn(a[0], b[0], q, qs, out, T, hq, scale, causal, window, mq_, mkv, scr, sb, None)


def sample(l=FAKE, stride=100, M=2, V=100, t=None, k=None, p=None, m=None, u=FAKE, ids=FAKE, probs=FAKE, scr=FAKE, sb=BIG):
    return mq.load().mq_sample(l, stride, M, V, t, k, p, m, u, ids, probs, scr, sb, None)


def test_cache_sizes():
    size = mq.kv_cache_bytes
    assert size(mq.Q4_0, 1, 16, 1, 128) == 2 * 16 * (64 + 8)
    assert size(mq.Q8_0, 10, 256, 4, 64) == 10 * 4 * 2 * 256 * (64 + 4)
    assert size(mq.Q4_0, 1 << 20, 64, 8, 256) == (1 << 20) * 8 * 2 * 64 * (128 + 16)
    for bad in ((mq.Q4_1, 1, 16, 1, 128), (mq.Q4_0, 0, 16, 1, 128), (mq.Q4_0, 1, 8, 1, 128), (mq.Q4_0, 1, 48, 1, 128),
                (mq.Q4_0, 1, 512, 1, 128), (mq.Q4_0, 1, 16, 0, 128), (mq.Q4_0, 1, 16, 257, 128), (mq.Q4_0, 1, 16, 1, 96),
                (mq.Q4_0, (1 << 28) + 1, 16, 1, 128)):
        assert size(*bad) == 0, bad
    for t in (mq.Q4_0, mq.Q8_0):
        for page in (16, 32, 64, 128, 256):
            for dim in (64, 128, 256):
                assert size(t, 3, page, 5, dim) == 15 * ko.chunk_bytes(t, page, dim)


@pytest.mark.parametrize("call,name", [(append, "mq_kv_append"), (read, "mq_kv_read"), (attn, "mq_attn")])
def test_cache_and_sequences_refused(call, name):
    for bad in (cache(data=None), cache(pages=0), cache(heads=-1)):
        assert call(c=bad) == -1 and name in mq.last_error()
    for bad in (seqs(q_start=None), seqs(kv_len=None), seqs(table=None), seqs(B=0), seqs(width=0)):
        assert call(s=bad) == -1 and name in mq.last_error()
    assert call(T=0) == -1 and call(T=-4) == -1
    for t in (mq.Q4_K, mq.Q4_1, mq.Q8_0 | mq.REPACKED, 0, -2):
        assert call(c=cache(t=t)) == -3
    for bad in (cache(page=24), cache(page=8), cache(page=512), cache(page=0), cache(dim=96), cache(dim=0), cache(heads=257),
                cache(pages=(1 << 28) + 1)):
        assert call(c=bad) == -2
    assert call(s=seqs(B=65537)) == -2 and call(T=(1 << 20) + 1) == -2 and call(s=seqs(width=(1 << 25) + 1)) == -2
    assert call(c=cache(data=FAKE + 8)) == -5
    for bad in (seqs(q_start=FAKE + 2), seqs(kv_len=FAKE + 1), seqs(table=FAKE + 2)):
        assert call(s=bad) == -5


def test_append_refusals():
    lib = mq.load()
    rest = (FAKE, 1024, FAKE, 512, FAKE, 512, FAKE, 1024, 5, 8, None, None, 1e-6, 1, FAKE, 128, None, None)
    assert lib.mq_kv_append(None, seqs()[0], *rest) == -1 and lib.mq_kv_append(cache()[0], None, *rest) == -1
    assert append(k=None) == -1 and append(v=None) == -1
    assert append(q=None) == -1 and append(out=None) == -1 and append(hq=0) == -1 and append(hq=-2) == -1
    assert append(q=None, out=None, hq=4) == -1
    assert append(rope=3) == -1 and append(rope=-1) == -1 and append(f=None) == -1
    assert append(rope=0) == -1 and append(rope=0, f=None) == -1 and append(rope=0, f=None, rot=0, pos=FAKE) == -1
    assert append(eps=-1.0) == -1 and append(eps=float("nan")) == -1
    assert append(rot=0) == -2 and append(rot=130) == -2 and append(rot=7) == -2 and append(hq=257, qs=1 << 20) == -2
    assert append(qs=1020) == -2 and append(qs=1026) == -2 and append(os_=512) == -2 and append(ks=508) == -2
    assert append(vs=513) == -2 and append(ks=(1 << 31) + 4) == -2
    assert append(os_=2048) == -1       # q_out is q, with another stride
    assert append(q=FAKE + 4) == -5 and append(out=FAKE + 8) == -5 and append(k=FAKE + 4) == -5 and append(v=FAKE + 8) == -5
    assert append(qn=FAKE + 2) == -5 and append(kn=FAKE + 1) == -5 and append(f=FAKE + 2) == -5 and append(pos=FAKE + 3) == -5
    assert "mq_kv_append" in mq.last_error()


def test_read_refusals():
    assert read(k=None, v=None) == -1 and read(k=FAKE + 4) == -5 and read(v=FAKE + 8) == -5


def test_attn_sizes_and_refusals():
    size = mq.attn_scratch_bytes
    for bad in ((mq.Q4_K, 1, 8, 4, 128, 1, 100), (mq.Q4_0, 0, 8, 4, 128, 1, 100), (mq.Q4_0, 1, 9, 4, 128, 1, 100),
                (mq.Q4_0, 1, 8, 0, 128, 1, 100), (mq.Q4_0, 1, 8, 4, 80, 1, 100), (mq.Q4_0, 1, 8, 4, 128, 0, 100),
                (mq.Q4_0, 1, 8, 4, 128, 1, 0), (mq.Q4_0, 1, 512, 4, 128, 1, 100), (mq.Q4_0, 1, 8, 4, 128, 1, (1 << 30) + 1)):
        assert size(*bad) == 0, bad
    assert attn(out=None) == -1 and attn(scr=None) == -1 and attn(q=None) == -1
    assert attn(hq=0) == -1 and attn(mq_=0) == -1 and attn(mkv=0) == -1
    assert attn(window=-1) == -1 and attn(window=5, causal=0) == -1 and attn(window=(1 << 30) + 1) == -1
    assert attn(hq=6) == -2 and attn(hq=512, qs=1 << 20) == -2 and attn(mq_=(1 << 20) + 1) == -2 and attn(mkv=(1 << 30) + 1) == -2
    assert attn(qs=1020) == -2 and attn(qs=1025) == -2
    assert attn(q=FAKE + 4) == -5 and attn(out=FAKE + 4) == -5 and attn(scr=FAKE + 8) == -5
    # workgroups of 256 threads, at most 2^32 of them: 65535 sequences of 256 heads fit, 65536 do not
    assert size(mq.Q4_0, 65536, 256, 256, 64, 1, 100) == 0 and size(mq.Q4_0, 65535, 256, 256, 64, 1, 100) > 0
    assert size(mq.Q4_0, 64, 64, 8, 128, 1 << 20, 100) == 0 and size(mq.Q4_0, 31, 64, 8, 128, 1 << 20, 100) > 0
    assert size(mq.Q4_0, 31, 64, 8, 256, 1 << 20, 100) == 0 and size(mq.Q4_0, 15, 64, 8, 256, 1 << 20, 100) > 0
    need = size(mq.Q4_0, 3, 8, 4, 128, 5, 1 << 20)
    if need:
        assert attn(mkv=1 << 20, sb=need - 1) == -4 and "scratch" in mq.last_error()


def test_attn_scale_that_is_not_finite_is_refused():
    for bad in (float("nan"), float("inf"), -float("inf"), 1e39):        # (1e39 is an infinity in f32)
        assert attn(scale=bad) == -1 and "mq_attn: scale=" in mq.last_error()
    for good in (0.0, -0.0, -2.5, 3.4e38, 1e-45):
        assert attn(scale=good, sb=0) == -4                              # (the next check: no scratch)


def test_sample_sizes_and_refusals():
    size = mq.sample_scratch_bytes
    assert size(0, 100) == size(1, 0) == size(1, (1 << 20) + 1) == size((1 << 20) + 1, 8) == 0
    for name in ("l", "u", "ids", "scr"):
        assert sample(**{name: None}) == -1, name
    assert sample(M=0) == -1 and sample(V=-1) == -1
    assert sample(V=(1 << 20) + 1, stride=1 << 21) == -2 and sample(M=(1 << 20) + 1) == -2
    assert sample(stride=99) == -2 and sample(stride=(1 << 31) + 1) == -2
    for name in ("l", "t", "k", "p", "m", "u", "ids", "probs"):
        assert sample(**{name: FAKE + 2}) == -5, name
    assert sample(scr=FAKE + 4) == -5 and "mq_sample" in mq.last_error()
    need = size(3, 152064)
    if need:
        assert sample(M=3, V=152064, stride=152064, sb=need - 1) == -4


def test_binding_refusals():
    import torch
    z = lambda *s, t=torch.float32: torch.zeros(s, dtype=t)   # noqa: E731
    size = mq.kv_cache_bytes(mq.Q4_0, 4, 16, 2, 64)
    data = z(size, t=torch.uint8)
    c = mq.KVCache(data, mq.Q4_0, 4, 16, 2, 64)
    i32 = lambda *s: z(*s, t=torch.int32)   # noqa: E731
    s = mq.KVSeqs(i32(4), i32(3), i32(3, 2))

    def refused(code, f, *a, **k):
        with pytest.raises(mq.MQError) as e:
            f(*a, **k)
        assert e.value.code == code, e.value

    refused(-4, mq.KVCache, data[:-1], mq.Q4_0, 4, 16, 2, 64)
    refused(-3, mq.KVCache, data, mq.Q4_K, 4, 16, 2, 64)
    refused(-2, mq.KVCache, data, mq.Q4_0, 4, 17, 2, 64)
    refused(-1, mq.KVCache, torch.zeros(2 * size, dtype=torch.uint8)[::2], mq.Q4_0, 4, 16, 2, 64)
    refused(-1, mq.KVSeqs, i32(4), i32(3), i32(6))
    refused(-4, mq.KVSeqs, i32(3), i32(3), i32(3, 2))
    refused(-4, mq.KVSeqs, i32(4), i32(4), i32(3, 2))
    refused(-1, mq.KVSeqs, i32(4).long(), i32(3), i32(3, 2))
    k, q = z(5, 2, 64), z(5, 4, 64)
    refused(-2, mq.kv_append, c, s, z(5, 3, 64), z(5, 2, 64))
    refused(-2, mq.kv_append, c, s, k, z(4, 2, 64))
    refused(-2, mq.kv_append, c, s, k, k, q=z(5, 4, 32))
    refused(-1, mq.kv_append, c, s, k.double(), k)
    refused(-1, mq.kv_append, c, s, z(5, 64, 2).transpose(1, 2), k)
    refused(-1, mq.kv_append, c, s, k, k, q_out=q)
    refused(-4, mq.kv_append, c, s, k, k, k_norm=z(32))
    refused(-1, mq.kv_append, c, s, k, k, pos=z(5))
    refused(-6, mq.kv_append, c, s, k, k)                   # CPU tensors
    refused(-6, mq.kv_read, c, s, 5)
    refused(-1, mq.attn, c, s, q.half())
    refused(-2, mq.attn, c, s, z(5, 4, 128))
    refused(-4, mq.attn, c, s, q, out=z(5, 4, 32))
    refused(-6, mq.attn, c, s, q)
    u = z(3)
    refused(-1, mq.sample, z(3, 10).half(), u)
    refused(-1, mq.sample, z(10, 3).t(), u)
    refused(-4, mq.sample, z(3, 10), z(2))
    refused(-1, mq.sample, z(3, 10), u, top_k=z(3))
    refused(-4, mq.sample, z(3, 10), u, min_p=z(4))
    refused(-6, mq.sample, z(3, 10), u)


@pytest.mark.parametrize("t", [mq.Q4_0, mq.Q8_0])
@pytest.mark.parametrize("page,dim", [(16, 64), (32, 128), (64, 256), (256, 64)])
def test_layout_covers_every_bit_once(t, page, dim):
    bits = ko.BITS[t]
    k, v, ks, vs, a, b = ko.places(t, page, dim)
    row = page * dim * bits // 8
    used = np.zeros((ko.chunk_bytes(t, page, dim), 8), int)
    for byte, shift in ((k, ks), (v, vs)):
        for i in range(bits):
            np.add.at(used, (byte.ravel(), shift.ravel() + i), 1)
    assert (used[:2 * row] == 1).all() and (used[2 * row:] == 0).all()
    assert k.max() < row <= v.min() and v.max() < 2 * row
    scales = np.concatenate([np.unique(a), np.unique(b)])
    assert (scales == 2 * row + 2 * np.arange(2 * page * dim // 32)).all()
    for w in (k, v):        # no byte of two tokens
        owner = np.full(2 * row, -1)
        for tok in range(page):
            assert (owner[w[tok]] == -1).all()
            owner[w[tok]] = tok


def test_layout_by_hand():
    """Dimension 32 b + 8 g + n of a 4-bit key; dimension 64 i + 16 j + c of a 4-bit value; 128 dimensions."""
    k, v, ks, vs, a, b = ko.places(mq.Q4_0, 32, 128)
    assert (k[0, 0], ks[0, 0]) == (0, 0) and (k[0, 1], ks[0, 1]) == (0, 4) and k[0, 7] == 3
    assert k[0, 32] == 4 and k[0, 8] == 16 and k[0, 127] == 63 and k[1, 0] == 64
    base = 32 * 64
    assert v[0, 0] == base and (v[0, 16], vs[0, 16]) == (base, 4) and v[0, 32] == base + 1
    assert v[0, 64] == base + 4 and v[1, 0] == base + 2 and v[2, 0] == base + 8 and v[0, 1] == base + 16
    assert v[4, 0] == base + 256 and v[16, 0] == base + 1024
    assert a[0, 0] == 2 * base and a[0, 127] == 2 * base + 6 and a[1, 0] == 2 * base + 8 and b[0, 0] == 2 * base + 256


def test_quantizer_by_hand():
    x = np.zeros(32, np.float32)
    x[3], x[7], x[9] = -8.0, 8.0, 3.5
    d, c = ko.quantize(x, mq.Q4_0)             # the first of largest magnitude is -8: d = 1
    assert d.view(np.float16)[0] == 1.0 and c[3] == 0 and c[7] == 15 and c[9] == 12 and c[0] == 8   # 3.5 + 8 is even at 12
    x[3] = 0.0
    d, c = ko.quantize(x, mq.Q4_0)             # now 8: d = -1
    assert d.view(np.float16)[0] == -1.0 and c[7] == 0 and c[9] == 4 and (ko.values(d, c, mq.Q4_0)[[7, 9]] == [8.0, 4.0]).all()
    d, c = ko.quantize(np.arange(-127, 127, 8).astype(np.float32), mq.Q8_0)
    assert d.view(np.float16)[0] == 1.0 and (c == np.arange(-127, 127, 8) + 128).all()
    for bad in (np.nan, np.inf):
        x[1] = bad
        for t in (mq.Q4_0, mq.Q8_0):
            d, c = ko.quantize(x, t)
            assert np.isnan(d.view(np.float16)).all() and (c == ko.OFFSET[t]).all()
    d, c = ko.quantize(np.zeros(64, np.float32), mq.Q4_0)
    assert (c == 8).all() and (ko.values(d, c, mq.Q4_0) == 0).all()


def test_rotation_by_hand():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 1], x[0, 0, 2] = 1.0, 2.0, 5.0
    quarter = np.array([np.pi / 2, 0.0])
    y = ko.rotated(x, [1], quarter, 1)          # pairs (0, 2), (1, 3): the first turned by 90 degrees
    assert np.allclose(y[0, 0, :4], [-5, 2, 1, 0])
    y = ko.rotated(x, [1], quarter, 2)          # pairs (0, 1), (2, 3)
    assert np.allclose(y[0, 0, :4], [-2, 1, 5, 0])


def test_sampling_by_hand():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))      # e = 1/4, 1, 1/2, 1/4
    assert ko.sample(l, 0.0)[0] == 0 and ko.sample(l, 0.124)[0] == 0 and ko.sample(l, 0.126)[0] == 1
    assert ko.sample(l, 0.99)[0] == 3 and ko.sample(l, 0.7)[0] == 2
    i, p = ko.sample(l, 0.9, top_k=2)
    assert i == 2 and abs(p - 1 / 3) < 1e-12
    assert ko.sample(l, 0.99, top_p=0.5)[0] == 1                # 1 of 2 is half of the mass
    assert ko.sample(l, 0.99, top_p=0.51)[0] == 2
    assert ko.sample(l, 0.99, top_k=3)[0] == 2 and ko.sample(l, 0.01, top_k=3)[0] == 0   # of the two equal ones the first
    assert ko.sample(l, 0.99, min_p=0.4)[0] == 2 and ko.sample(l, 0.99, min_p=5.0) == (1, 1.0)
    assert ko.sample(l, 0.5, T=0.0) == (1, 1.0)
    assert ko.sample([-np.inf, np.nan], 0.5) == (-1, 0.0)
    assert ko.sample([np.nan, 1.0, -np.inf], 0.99) == (1, 1.0)
    assert ko.sample([np.inf, 0.0, np.inf], 0.6) == (2, 0.5)


def test_calls_without_init_are_refused():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a device is there")
    assert append() in (-6, -8) and read() in (-6, -8) and attn() in (-6, -8) and sample() in (-6, -8)
