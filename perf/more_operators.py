"""Timed cases of the operators between the products of a decoder layer and after its vocabulary head:
norm, rotation and append of keys and values to a paged cache held in blocks of 4 or 8 bits, attention over
that cache, and sampling.

``own`` False: the operators from elementary torch operations; ``own`` True: the framework's calls.
"""

import random

import numpy as np
import torch

own = False

BITS = {"q4_0": 4, "q8_0": 8}


# ------------------------------------------------------------------ the cases

def _append(**kw):
    return dict(dict(op="append", seqs=1, tokens=1, past=0, Hq=28, Hkv=4, D=128, page=64, type="q4_0", norm=False,
                     rope="half", rot=0, fused=True, idle=False), **kw)


def _attn(**kw):
    return dict(dict(op="attn", seqs=1, tokens=1, kv=1024, ragged=False, Hq=28, Hkv=4, D=128, page=64, type="q4_0",
                     causal=True, window=0, idle=False), **kw)


def _sample(**kw):
    return dict(dict(op="sample", M=1, V=152064, kind="filters", masked=False), **kw)


def listed():
    return [
        # decode: one token of the 7B's layer, its q, k and v in one product's row
        _append(name="append 1 token 28/4x128 q4_0", past=1023),
        # seven sequences, a few tokens each (drafts to verify), normed heads of 64 of the 0.5B in 8 bits, small pages
        _append(name="append 7x<=6 tokens 14/2x64 q8_0 normed", seqs=7, tokens=6, past=301, Hq=14, Hkv=2, D=64, page=16,
                type="q8_0", norm=True, fused=False, idle=True),
        # a prompt of three sequences through the 14B's heads
        _append(name="append 3x<=1365 tokens 40/8x128 q4_0 normed", seqs=3, tokens=1365, Hq=40, Hkv=8, page=64, norm=True),
        # decode: one token of the 0.5B over a short odd context
        _attn(name="decode 1x777 14/2x64 q4_0", kv=777, Hq=14, Hkv=2, D=64, page=16),
        # decode: one token of the 7B over a long context
        _attn(name="decode 1x32768 28/4x128 q4_0", kv=32768),
        # decode: 64 sequences of the 14B of all lengths up to 8192
        _attn(name="decode 64x<=8192 40/8x128 q4_0", seqs=64, kv=8192, ragged=True, Hq=40, Hkv=8),
        # verification of drafts: five sequences, up to seven tokens each, in 8 bits, a sliding window
        _attn(name="verify 5x<=7 over <=4099 28/4x128 q8_0 window", seqs=5, tokens=7, kv=4099, ragged=True, page=32,
              type="q8_0", window=2048, idle=True),
        # a prompt chunk of the 7B behind a long context
        _attn(name="prefill 512 over 8192 28/4x128 q4_0", tokens=512, kv=8192),
        # a whole prompt of the 14B
        _attn(name="prefill 2048 over 2048 40/8x128 q4_0", tokens=2048, kv=2048, Hq=40, Hkv=8),
        # one decoded token, every filter
        _sample(name="sample 1x152064 top-k top-p min-p"),
        # nine sequences over a small odd vocabulary, top-p over a flat distribution
        _sample(name="sample 9x32003 top-p", M=9, V=32003, kind="nucleus"),
        # 128 sequences decoded together, each with settings of its own, greedy ones among them, masked tokens
        _sample(name="sample 128x152064 mixed", M=128, kind="mixed", masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


HEADS = [(14, 2), (28, 4), (40, 8), (8, 8), (16, 1), (12, 4), (9, 3)]


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "sample"])
    if op == "sample":
        return _sample(M=_log(rng, 1, 128), V=_log(rng, 500, 152064), kind=rng.choice(["filters", "nucleus", "mixed", "plain"]),
                       masked=rng.random() < 0.3)
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128, 128, 256])
    both = dict(Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), type=rng.choice(["q4_0", "q4_0", "q8_0"]),
                idle=rng.random() < 0.3)
    seqs = _log(rng, 1, 48)
    if op == "append":
        return _append(seqs=seqs, tokens=_log(rng, 1, max(1, (1 << 23) // (Hq * D * seqs))), past=_log(rng, 1, 4096) - 1,
                       norm=rng.random() < 0.5, rope=rng.choice(["half", "half", "interleaved", "none"]),
                       rot=rng.choice([0, 0, D // 2]), fused=rng.random() < 0.5, **both)
    if rng.random() < 0.6:      # decode, or a few tokens at a time
        kv = _log(rng, 1, max(64, min(32768, (1 << 26) // (seqs * Hkv * D))))
        tokens = rng.choice([1, 1, 1, 2, 5, 8])
    else:
        seqs = rng.choice([1, 1, 2, 5])
        tokens = _log(rng, 9, 700)
        kv = tokens + _log(rng, 1, 4096) - 1
    return _attn(seqs=seqs, tokens=min(tokens, kv), kv=kv, ragged=rng.random() < 0.6, causal=rng.random() < 0.85,
                 window=rng.choice([0, 0, _log(rng, 16, 2048)]), **both)


def _plan(case):
    """(tokens, cached length with them) of each sequence: of the case alone."""
    rng = random.Random(case["seqs"] * 1000003 + case["tokens"])
    n, kv = [], []
    for b in range(case["seqs"]):
        if case["idle"] and b % 4 == 2:     # a slot that no sequence holds
            n.append(0), kv.append(0)
            continue
        ragged = case.get("ragged", True) and b > 0
        n.append(rng.randint(1, case["tokens"]) if ragged else case["tokens"])
        if case["op"] == "append":
            kv.append(n[-1] + (rng.randint(0, case["past"]) if b else case["past"]))
        else:
            kv.append(rng.randint(n[-1], case["kv"]) if ragged else case["kv"])
    return n, kv


def _window(case):
    return case["window"] if case["causal"] else 0


def work(case):
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        return {"bytes": 4 * M * V + 28 * M, "flops": 4 * M * V}
    n, kv = _plan(case)
    T, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], case["D"]
    row = D * BITS[case["type"]] // 8 + D // 16      # bytes of a head's key, or value
    if case["op"] == "append":
        # the rows, the rotated queries, the cache written; read back, as f32
        return {"bytes": 4 * T * D * (Hq + 2 * Hkv) + 4 * T * D * Hq + 2 * (2 * T * Hkv * row) + 4 * T * D * 2 * Hkv,
                "flops": T * D * (8 * Hq + 12 * Hkv)}
    W = _window(case)
    pairs = keys = 0
    for a, l in zip(n, kv):
        if not case["causal"]:
            seen = a * l
            low = 0
        else:
            i = np.arange(l - a, l, dtype=np.int64)
            seen = int(np.minimum(i + 1, W).sum() if W else (i + 1).sum())
            low = max(0, l - a + 1 - W) if W else 0
        pairs += seen
        keys += (l - low) if a else 0
    return {"bytes": 2 * keys * Hkv * row + 8 * T * Hq * D, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ inputs

def _chunk_bytes(case):
    return 2 * case["page"] * (case["D"] * BITS[case["type"]] // 8 + case["D"] // 16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device="cuda", generator=gen)

    s = {"case": case}
    if case["op"] == "sample":
        M, V = case["M"], case["V"]
        z = normal(M, V) * (1.5 if case["kind"] == "nucleus" else 2.5)
        z[:, :max(1, V // 1000)] += 4.0      # the words that fit here
        z = z.gather(1, torch.argsort(uniform(1, V), 1).expand(M, V))
        if case["masked"]:                   # a grammar's tokens alone
            z = torch.where(uniform(M, V) < 0.3, -torch.inf, z)
        s["logits"] = z.contiguous()
        s["u"] = uniform(M)
        one = torch.ones(M, device="cuda")
        s["temperature"] = s["top_k"] = s["top_p"] = s["min_p"] = None
        if case["kind"] == "filters":
            s["temperature"], s["top_k"] = 0.8 * one, torch.full((M,), 40, dtype=torch.int32, device="cuda")
            s["top_p"], s["min_p"] = 0.95 * one, 0.05 * one
        elif case["kind"] == "nucleus":
            s["top_p"] = 0.9 * one
        elif case["kind"] == "mixed":
            s["temperature"] = torch.where(uniform(M) < 0.2, 0.0, 0.5 + uniform(M))
            s["top_k"] = torch.where(uniform(M) < 0.5, 0, (1 + 200 * uniform(M)).int()).int()
            s["top_p"] = torch.where(uniform(M) < 0.4, 1.0, 0.7 + 0.3 * uniform(M))
            s["min_p"] = torch.where(uniform(M) < 0.5, 0.0, 0.1 * uniform(M))
        s["scratch"] = torch.zeros((32 << 20) + 8 * M * V, dtype=torch.uint8, device="cuda")
        return s

    n, kv = _plan(case)
    T, Hq, Hkv, D, page = sum(n), case["Hq"], case["Hkv"], case["D"], case["page"]
    per = [-(-l // page) for l in kv]
    wide = max(max(per), 1) + 1
    pages = sum(per) + 3
    order = torch.randperm(pages, device="cuda", generator=gen).int()
    table = torch.full((case["seqs"], wide), -1, dtype=torch.int32)
    at = torch.tensor([0] + per).cumsum(0)
    rows = torch.arange(wide)[None, :]
    table = torch.where(rows < torch.tensor(per)[:, None], at[:-1, None] + rows, -1).cuda()
    s["table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).int().contiguous()
    s["q_start"] = torch.tensor([0] + n).cumsum(0).int().cuda()
    s["kv_len"] = torch.tensor(kv).int().cuda()
    s["max_q"], s["max_kv"], s["pages"] = max(max(n), 1), max(max(kv), 1), pages
    if case["op"] == "append":
        width = (Hq + 2 * Hkv) * D
        if case["fused"]:       # one product's rows
            x = normal(T, width)
            s["q"], s["k"], s["v"] = (p.unflatten(1, (-1, D)) for p in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        else:
            s["q"], s["k"], s["v"] = normal(T, Hq, D), normal(T, Hkv, D), normal(T, Hkv, D)
        s["q_norm"] = 1.0 + 0.1 * normal(D) if case["norm"] else None
        s["k_norm"] = 1.0 + 0.1 * normal(D) if case["norm"] else None
        rot = case["rot"] or D
        freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        s["inv_freq"] = None if case["rope"] == "none" else freq.float().cuda()
        s["data"] = torch.zeros(pages * Hkv * _chunk_bytes(case), dtype=torch.uint8, device="cuda")
        return s
    s["q"] = normal(T, Hq, D)
    chunk = _chunk_bytes(case)
    codes = chunk - 4 * page * (D // 32)
    lo, hi = (0, 256) if case["type"] == "q4_0" else (1, 256)
    data = torch.randint(lo, hi, (pages, Hkv, chunk), dtype=torch.uint8, device="cuda", generator=gen)
    unit = 0.22 if case["type"] == "q4_0" else 0.0136      # values of a deviation of about 1
    d = unit * (0.6 + 0.8 * uniform(pages, Hkv, 2 * page * (D // 32)))
    if case["type"] == "q4_0":       # (the sign is that of the block's largest value)
        d = torch.where(uniform(*d.shape) < 0.5, -d, d)
    data[:, :, codes:] = d.half().view(torch.uint8)
    s["data"] = data.view(-1)
    s["scratch"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain form

def _token_rows(s):
    """Sequence and position in the cache of each token, in 64-bit integers."""
    q_start, kv = s["q_start"].long(), s["kv_len"].long()
    T = s["q"].shape[0]
    t = torch.arange(T, device=q_start.device)
    b = (torch.searchsorted(q_start, t, right=True) - 1).clamp(0, kv.numel() - 1)
    return b, kv[b] - (q_start[b + 1] - t)


def _normed(x, w):
    x = x.double()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + float(np.float32(1e-6))) * w.double()


def _rotated(x, angle, rope):
    if rope == "none":
        return x
    rot = 2 * angle.shape[-1]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    y, rest = x[..., :rot], x[..., rot:]
    if rope == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = y[..., 0::2], y[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _held(x, t):
    """f32 rows as the values that blocks of 32 hold."""
    b = x.unflatten(-1, (-1, 32))
    if t == "q4_0":
        m = torch.gather(b, -1, b.abs().argmax(-1, keepdim=True))
        d = (m / -8.0).half().float()
        code = torch.clamp(torch.round(b / d) + 8.0, 0.0, 15.0) - 8.0
    else:
        d = (b.abs().amax(-1, keepdim=True) / 127.0).half().float()
        code = torch.clamp(torch.round(b / d), -127.0, 127.0)
    return torch.where(d == 0, 0.0, code * d).flatten(-2)


def _plain_append(s):
    c = s["case"]
    _, pos = _token_rows(s)
    angle = None        # in 64 bits: far positions, and keys next to a border of their codes
    if c["rope"] != "none":
        angle = pos.double()[:, None] * s["inv_freq"].double()[None, :]
    q = _rotated(_normed(s["q"], s["q_norm"]), angle, c["rope"]).float()
    k = _rotated(_normed(s["k"], s["k_norm"]), angle, c["rope"]).float()
    return {"q": q, "k": _held(k, c["type"]), "v": _held(s["v"].float(), c["type"])}


def _cached(s, pages):
    """K and V, f32 [..., page, Hkv, D], of page numbers [...]."""
    c = s["case"]
    D, P, Hkv, nb = c["D"], c["page"], c["Hkv"], c["D"] // 32
    raw = s["data"].view(s["pages"], Hkv, -1)[pages]
    size = P * D * BITS[c["type"]] // 8
    k, v, ks, vs = raw.split([size, size, 2 * P * nb, 2 * P * nb], -1)
    scale = [x.contiguous().view(torch.float16).float().unflatten(-1, (P, nb, 1)) for x in (ks, vs)]
    lead = k.shape[:-1]
    if c["type"] == "q4_0":
        kc = k.reshape(*lead, P, 4, nb, 4)
        kc = torch.stack([kc & 15, kc >> 4], -1).flatten(-2).transpose(-3, -2)              # block, eighth, value
        vc = v.reshape(*lead, P // 16, 4, 16, 2, D // 64, 2, 2)                             # tile g c pair i half byte
        vc = torch.stack([vc & 15, vc >> 4], -1)
        a = len(lead)
        vc = vc.permute(*range(a), a, a + 1, a + 3, a + 5, a + 4, a + 6, a + 7, a + 2)
        off = 8.0
    else:
        kc = k.reshape(*lead, P, 4, nb, 8).transpose(-3, -2)
        vc = v.reshape(*lead, P // 16, 4, 16, 2, nb, 2, 2)                                  # tile g c pair i half j
        a = len(lead)
        vc = vc.permute(*range(a), a, a + 1, a + 3, a + 5, a + 4, a + 6, a + 2)
        off = 128.0
    kf = (kc.reshape(*lead, P, nb, 32).float() - off) * scale[0]
    vf = (vc.reshape(*lead, P, nb, 32).float() - off) * scale[1]
    return kf.flatten(-2).transpose(-3, -2), vf.flatten(-2).transpose(-3, -2)


def _plain_attn(s):
    c = s["case"]
    q, D, Hq, Hkv, B = s["q"], c["D"], c["Hq"], c["Hkv"], c["seqs"]
    T, G, N, L = q.shape[0], Hq // Hkv, s["max_q"], s["max_kv"]
    np_ = -(-L // c["page"])
    k, v = (x.transpose(2, 3).transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :L]
            for x in _cached(s, s["table"][:, :np_].clamp(min=0).long()))
    start, kv = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(N, device=q.device)
    rows = torch.where(i < n[:, None], start[:-1, None] + i, T)          # T: no token
    qp = torch.cat([q, q.new_zeros(1, Hq, D)])[rows]                     # [B, N, Hq, D]
    qp = qp.view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    S = torch.matmul(qp, k.transpose(2, 3)).view(B, Hkv, N, G, L) * (1.0 / D ** 0.5)
    at, key = (kv - n)[:, None, None] + i[:, None], torch.arange(L, device=q.device)
    see = (key < kv[:, None, None]) & (i[:, None] < n[:, None, None])
    if c["causal"]:
        see = see & (key <= at)
    if _window(c):
        see = see & (key > at - _window(c))
    see = see[:, None, :, None, :]
    S = torch.where(see, S, -torch.inf)
    top = S.amax(-1, keepdim=True)
    e = torch.where(see, torch.exp(S - torch.where(torch.isinf(top), 0.0, top)), 0.0)
    total = e.sum(-1, keepdim=True)
    e = (e / torch.where(total > 0, total, 1.0)).view(B, Hkv, N * G, L)
    o = torch.matmul(e, torch.where((key < kv[:, None])[:, None, :, None], v, 0.0))
    o = o.view(B, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B * N, Hq, D)
    out = q.new_zeros(T + 1, Hq, D)
    return out.index_copy_(0, rows.view(-1).clamp(max=T), o)[:T]


def _plain_sample(s):
    z, u = s["logits"].double(), s["u"].double()       # in 64 bits: a draw next to a border has to fall the same way
    M, V = z.shape
    one = torch.ones_like(u)
    T = one if s["temperature"] is None else s["temperature"].double()
    k = torch.full_like(u, V) if s["top_k"] is None else torch.where(s["top_k"] > 0, s["top_k"], V).double()
    p = one if s["top_p"] is None else s["top_p"].double()
    m = 0.0 * one if s["min_p"] is None else s["min_p"].double()
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    x = (zs[:, :1] - zs) / torch.where(T > 0, T, 1.0)[:, None]
    e = torch.exp(-x)
    rank = torch.arange(V, device=z.device)
    keep = rank < torch.where(T > 0, k, 1.0)[:, None]
    e = torch.where(keep, e, 0.0)
    before = e.cumsum(1) - e
    cut = torch.where(p < 1.0, p, torch.inf)[:, None] * e.sum(1, keepdim=True)
    keep = keep & ((before < cut) | (rank == 0)) & (e >= m[:, None])
    e = torch.where(keep, e, 0.0)
    w = torch.zeros_like(z).scatter_(1, order, e)
    total = w.sum(1, keepdim=True)
    ids = ((w.cumsum(1) > u[:, None] * total) & (w > 0)).int().argmax(1)
    return {"ids": ids.int(), "probs": (torch.gather(w, 1, ids[:, None]) / total)[:, 0].float()}


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from block_quantized_matmul_mq_amd import mq
    c = s["case"]
    if c["op"] == "sample":
        if "ready" not in s:
            mq.init(s["logits"].device.index or 0)
            s["ready"] = True
        ids, probs = mq.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"], scratch=s["scratch"])
        return {"ids": ids, "probs": probs}
    if "cache" not in s:
        mq.init(s["q"].device.index or 0)
        s["cache"] = mq.KVCache(s["data"], {"q4_0": mq.Q4_0, "q8_0": mq.Q8_0}[c["type"]], s["pages"], c["page"],
                                c["Hkv"], c["D"])
        s["seqs"] = mq.KVSeqs(s["q_start"], s["kv_len"], s["table"])
    if c["op"] == "append":
        rope = {"half": mq.ROPE_HALF, "interleaved": mq.ROPE_INTERLEAVED, "none": mq.ROPE_NONE}[c["rope"]]
        q = mq.kv_append(s["cache"], s["seqs"], s["k"], s["v"], q=s["q"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                         eps=1e-6, rope=rope, inv_freq=s["inv_freq"])
        k, v = mq.kv_read(s["cache"], s["seqs"], s["q"].shape[0])
        return {"q": q, "k": k, "v": v}
    return mq.attn(s["cache"], s["seqs"], s["q"], causal=c["causal"], window=_window(c), max_q=s["max_q"],
                   max_kv=s["max_kv"], scratch=s["scratch"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits, from the definitions

def _exact_append(s):
    c = s["case"]
    D = c["D"]
    n, kv = _plan(c)
    pos = np.concatenate([np.arange(l - a, l) for a, l in zip(n, kv)])
    turn = np.ones((len(pos), D // 2), np.complex128)       # of pair j, or of dimensions that stay: 1
    rot = c["rot"] or D
    if c["rope"] != "none":
        turn = np.exp(1j * pos[:, None].astype(np.float64) * s["inv_freq"].cpu().numpy().astype(np.float64))
    first = np.arange(rot // 2) * (2 if c["rope"] == "interleaved" else 1)
    second = first + (1 if c["rope"] == "interleaved" else rot // 2)

    def through(x, w):
        x = x.cpu().numpy().astype(np.float64)
        if w is not None:
            x = x / np.sqrt(np.mean(x ** 2, -1, keepdims=True) + np.float64(np.float32(1e-6))) * w.cpu().numpy()
        if c["rope"] != "none":
            z = (x[..., first] + 1j * x[..., second]) * turn[:, None]
            x = x.copy()
            x[..., first], x[..., second] = z.real, z.imag
        return x

    def blocks(x):
        b = x.astype(np.float32).reshape(-1, 32)
        big = np.abs(b)
        if c["type"] == "q4_0":
            m = b[np.arange(len(b)), big.argmax(1)]
            d = (m / np.float32(-8)).astype(np.float16).astype(np.float32)[:, None]
            lo, hi = -8, 7
        else:
            d = (big.max(1) / np.float32(127)).astype(np.float16).astype(np.float32)[:, None]
            lo, hi = -127, 127
        code = np.rint(np.divide(b, d, out=np.zeros_like(b), where=d != 0)).clip(lo, hi)
        return (code.astype(np.float64) * d).reshape(x.shape)

    return {"q": through(s["q"], s["q_norm"]), "k": blocks(through(s["k"], s["k_norm"])),
            "v": blocks(s["v"].cpu().numpy())}


def _exact_rows(s, pages, count):
    """K and V, f64 [Hkv, count, D], of a sequence: every value fetched at its own byte."""
    c = s["case"]
    D, P, nb = c["D"], c["page"], c["D"] // 32
    dev = s["data"].device
    raw = s["data"].view(s["pages"], c["Hkv"], -1)
    tok, dim = torch.arange(count, device=dev)[:, None], torch.arange(D, device=dev)[None, :]
    page, t = pages.long()[tok // P], tok % P
    section = P * D * BITS[c["type"]] // 8
    tile, g, pair, half = t // 16, t % 16 // 4, t % 4 // 2, t % 2

    def fetch(at):
        return raw[page[:, :, None], torch.arange(c["Hkv"], device=dev), at[:, :, None]].permute(2, 0, 1).int()

    def halves(at):
        lo, hi = fetch(at), fetch(at + 1)
        bits = lo + 256 * hi
        frac, ex = (bits & 1023).double(), (bits >> 10) & 31
        mag = torch.where(ex == 0, frac * 2.0 ** -24, (1024.0 + frac) * torch.pow(2.0, (ex - 25).double()))
        return torch.where(bits >= 32768, -mag, mag)

    if c["type"] == "q4_0":
        r = dim % 8
        code = fetch(t * (D // 2) + 4 * (dim % 32 // 8 * nb + dim // 32) + r // 2)
        k = torch.where((r % 2 == 1).expand(count, D), code // 16, code % 16) - 8
        j = dim % 64 // 16
        code = fetch(section + tile * 8 * D + 4 * (((g * 16 + dim % 16) * 2 + pair) * (D // 64) + dim // 64) + 2 * half + j // 2)
        v = torch.where((j % 2 == 1).expand(count, D), code // 16, code % 16) - 8
    else:
        k = fetch(t * D + 8 * (dim % 32 // 8 * nb + dim // 32) + dim % 8) - 128
        v = fetch(section + tile * 16 * D + 4 * (((g * 16 + dim % 16) * 2 + pair) * nb + dim // 32) + 2 * half + dim % 32 // 16) - 128
    at = 2 * section + 2 * (t * nb + dim // 32)
    return k.double() * halves(at), v.double() * halves(at + 2 * P * nb)


def _exact_attn(s):
    c = s["case"]
    n, kv = _plan(c)
    G, D, W = c["Hq"] // c["Hkv"], c["D"], _window(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (a, l) in enumerate(zip(n, kv)):
        if a:
            k, v = _exact_rows(s, s["table"][b], l)
            key = torch.arange(l, device="cuda")
            for lo in range(0, a, 256):
                hi = min(a, lo + 256)
                q = s["q"][at + lo:at + hi].double().view(hi - lo, c["Hkv"], G, D).permute(1, 2, 0, 3).reshape(c["Hkv"], -1, D)
                score = (q @ k.transpose(1, 2).contiguous()) / D ** 0.5
                here = torch.arange(l - a + lo, l - a + hi, device="cuda").repeat(G)[:, None]
                hide = torch.zeros((G * (hi - lo), l), dtype=torch.bool, device="cuda")
                if c["causal"]:
                    hide |= key > here
                    if W:
                        hide |= key <= here - W
                score = score.masked_fill(hide, -torch.inf)
                o = torch.softmax(score, -1) @ v
                out[at + lo:at + hi] = o.view(c["Hkv"], G, hi - lo, D).permute(2, 0, 1, 3).reshape(hi - lo, -1, D)
        at += a
    return out


def _exact_sample(s):
    ids, probs = [], []

    def value(name, m, default):
        return default if s[name] is None else s[name][m].item()

    z, u = s["logits"].cpu().numpy().astype(np.float64), s["u"].cpu().numpy().astype(np.float64)
    for m in range(len(z)):
        T, k = value("temperature", m, 1.0), value("top_k", m, 0)
        p, low = value("top_p", m, 1.0), value("min_p", m, 0.0)
        order = np.argsort(-z[m], kind="stable")
        if T <= 0:
            ids.append(order[0]), probs.append(1.0)
            continue
        order = order[:k] if k > 0 else order
        e = np.exp((z[m][order] - z[m][order[0]]) / T)
        if p < 1:
            cum = np.cumsum(e)
            count = int(np.searchsorted(cum, p * cum[-1], side="left")) + 1
            order, e = order[:count], e[:count]
        order, e = order[e >= low], e[e >= low]
        by = np.argsort(order)
        order, e = order[by], e[by]
        order, e = order[e > 0], e[e > 0]
        cum = np.cumsum(e)
        j = min(int(np.searchsorted(cum, u[m] * cum[-1], side="right")), len(e) - 1)
        ids.append(order[j]), probs.append(e[j] / cum[-1])
    return {"ids": np.array(ids, dtype=np.int32), "probs": np.array(probs)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](s)
