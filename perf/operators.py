"""Timed cases of the feed-forward operators: mixture-of-experts routing, the expert layer for a few
tokens, and the block-quantized products with bias, activation, multiplier and residual in their
epilogue.

``own`` False: the operators from elementary torch operations; ``own`` True: the framework's calls.
"""

import numpy as np
import torch

own = False

# GGUF block types by name: values and bytes per block
BLOCKS = {"q4_0": (32, 18), "q4_1": (32, 20), "q5_0": (32, 22), "q5_1": (32, 24), "q8_0": (32, 34),
          "q4_K": (256, 144), "q5_K": (256, 176), "q6_K": (256, 210)}
GEMM_SCRATCH = 48 << 20     # bytes of workspace a program keeps for the prefill products
ACTS = ("none", "silu", "gelu_tanh", "gelu_erf", "relu")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the router of one decoded token, 64 experts: a few launches' worth of latency
        dict(name="route 1x2048 e64 k8", op="route", M=1, K=2048, E=64, k=8, score="softmax", norm=True, bias=False),
        # the router of a 512-token prompt chunk, sigmoid scores with a selection bias
        dict(name="route 512x4096 e128 k8", op="route", M=512, K=4096, E=128, k=8, score="sigmoid", norm=True, bias=True),
        # one decoded token through 8 of 64 small experts
        dict(name="moe m1 e64 q4_K", op="moe", M=1, E=64, k=8, K=2048, F=1024, gu="q4_K", down="q4_K", act="silu", residual=True, pad=False),
        # one decoded token through 4 of 32 larger experts, the down weights in 6 bits
        dict(name="moe m1 e32 q4_K q6_K", op="moe", M=1, E=32, k=4, K=4096, F=2048, gu="q4_K", down="q6_K", act="silu", residual=False, pad=False),
        # seven sequences decoded together, odd sizes in 8-bit weights, some choices dropped
        dict(name="moe m7 e60 q8_0", op="moe", M=7, E=60, k=4, K=2048, F=1408, gu="q8_0", down="q8_0", act="silu", residual=True, pad=True),
        # 48 sequences decoded together: nearly every expert is read
        dict(name="moe m48 e128 q4_K q6_K", op="moe", M=48, E=128, k=8, K=4096, F=1536, gu="q4_K", down="q6_K", act="silu", residual=True, pad=False),
        # decode: the small model's ffn_down with the residual stream added in place of a second launch
        dict(name="gemv 896x4864 q8_0", op="gemv", N=896, K=4864, type="q8_0", bias=True, act="none", mul=False, residual=True),
        # decode: the 7B ffn_gate whose epilogue makes silu(gate) * up
        dict(name="gemv 18944x3584 q4_K", op="gemv", N=18944, K=3584, type="q4_K", bias=False, act="silu", mul=True, residual=False),
        # decode: the 7B ffn_down with the residual
        dict(name="gemv 3584x18944 q6_K", op="gemv", N=3584, K=18944, type="q6_K", bias=False, act="none", mul=False, residual=True),
        # a handful of rows (a draft's verification) with bias and gelu
        dict(name="gemm 5x4864x896 q5_0", op="gemm", M=5, N=4864, K=896, type="q5_0", bias=True, act="gelu_tanh", mul=False, residual=False),
        # a ragged prompt chunk through the 14B ffn_down with the residual
        dict(name="gemm 333x5120x13824 q6_K", op="gemm", M=333, N=5120, K=13824, type="q6_K", bias=False, act="none", mul=False, residual=True),
        # a 512-token prompt chunk through the 7B ffn_gate: silu(gate) * up
        dict(name="gemm 512x18944x3584 q4_K", op="gemm", M=512, N=18944, K=3584, type="q4_K", bias=False, act="silu", mul=True, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "gemv", "gemm"])
    if op == "route":
        E = rng.choice([8, 16, 40, 60, 64, 128, 160, 256])
        return dict(op=op, M=_log(rng, 1, 512), K=32 * _log(rng, 8, 128), E=E, k=rng.randint(1, min(E, 8)),
                    score=rng.choice(["softmax", "sigmoid"]), norm=rng.random() < 0.7, bias=rng.random() < 0.4)
    if op == "moe":
        E = rng.choice([4, 8, 16, 32, 60, 64, 128])
        gu = rng.choice(["q4_K", "q4_K", "q5_K", "q6_K", "q8_0", "q4_0", "q5_1"])
        down = rng.choice([gu, "q6_K", "q8_0"])
        K = 256 * rng.randint(2, 16) if BLOCKS[gu][0] == 256 else 32 * rng.randint(16, 100)
        F = 256 * rng.randint(1, 6) if BLOCKS[down][0] == 256 else 32 * rng.randint(8, 40)
        return dict(op=op, M=_log(rng, 1, 48), E=E, k=rng.randint(1, min(E, 8)), K=K, F=F, gu=gu, down=down,
                    act=rng.choice(["silu", "silu", "gelu_tanh"]), residual=rng.random() < 0.5, pad=rng.random() < 0.3)
    t = rng.choice(list(BLOCKS))
    step = BLOCKS[t][0]
    K = step * max(1, _log(rng, 512, 14336) // step)
    ep = dict(type=t, bias=rng.random() < 0.5, act=rng.choice(ACTS), mul=rng.random() < 0.4, residual=rng.random() < 0.5)
    if op == "gemv":
        return dict(op=op, N=_log(rng, 512, 18944), K=K, **ep)
    return dict(op=op, M=_log(rng, 2, 512), N=_log(rng, 512, 5120), K=K, **ep)


def _nbytes(t, rows, K):
    v, b = BLOCKS[t]
    return rows * (K // v) * b


def work(case):
    op = case["op"]
    if op == "route":
        M, K, E, k = (case[n] for n in ("M", "K", "E", "k"))
        return {"bytes": 4 * (M * K + E * K + 2 * M * k), "flops": 2 * M * K * E}
    if op == "moe":
        M, K, F, E, k = (case[n] for n in ("M", "K", "F", "E", "k"))
        live = 0.875 if case["pad"] else 1.0
        experts = E * (1.0 - (1.0 - live * k / E) ** M)     # expected number of experts that some token chose
        per = 2 * _nbytes(case["gu"], F, K) + _nbytes(case["down"], K, F)
        return {"bytes": experts * per + 4 * M * K * (3 if case["residual"] else 2) + 8 * M * k,
                "flops": 6 * live * M * k * F * K}
    M, N, K = case.get("M", 1), case["N"], case["K"]
    rows = 1 + int(case["mul"]) + int(case["residual"])
    return {"bytes": _nbytes(case["type"], N, K) + 4 * (M * K + rows * M * N + (N if case["bias"] else 0)),
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _weights(t, rows, K, gen):
    """uint8 [rows, row bytes] of random blocks whose values have a deviation of about 0.02."""
    v, b = BLOCKS[t]
    nb = K // v
    raw = torch.randint(0, 256, (rows, nb, b), dtype=torch.uint8, device="cuda", generator=gen)
    jitter = 0.6 + 0.8 * torch.rand((rows, nb), device="cuda", generator=gen)

    def put(at, value):
        raw[..., at:at + 2] = value.half().unsqueeze(-1).view(torch.uint8)

    if t in ("q4_K", "q5_K"):
        d = jitter * (7.8e-5 if t == "q4_K" else 3.9e-5)
        put(0, d)
        put(2, d * (7.5 if t == "q4_K" else 15.5))
    elif t == "q6_K":
        put(208, jitter * 1.5e-5)
    elif t == "q8_0":
        put(0, jitter * 2.7e-4)
    else:
        d = jitter * (4.3e-3 if t[1] == "4" else 2.2e-3)
        put(0, d)
        if t.endswith("_1"):
            put(2, d * (-7.5 if t[1] == "4" else -15.5))
    return raw.view(rows, nb * b)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    s = {"case": case}
    op = case["op"]
    if op == "route":
        M, K, E = case["M"], case["K"], case["E"]
        s["X"] = normal(M, K)
        s["Wr"] = normal(E, K) * (2.0 / K ** 0.5)
        s["bias"] = normal(E) * 0.1 if case["bias"] else None
        s["scratch"] = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    elif op == "moe":
        M, K, F, E, k = (case[n] for n in ("M", "K", "F", "E", "k"))
        s["X"] = normal(M, K)
        s["Wg"] = _weights(case["gu"], E * F, K, gen)
        s["Wu"] = _weights(case["gu"], E * F, K, gen)
        s["Wd"] = _weights(case["down"], E * K, F, gen)
        s["residual"] = normal(M, K) if case["residual"] else None
        ids = torch.argsort(torch.rand((M, E), device="cuda", generator=gen), dim=1)[:, :k]
        if case["pad"]:     # choices that another device serves
            ids = torch.where(torch.rand((M, k), device="cuda", generator=gen) < 0.125, -1, ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        p = torch.rand((M, k), device="cuda", generator=gen) + 0.1
        s["wts"] = (p / p.sum(1, keepdim=True)).contiguous()
        s["scratch"] = torch.zeros((1 << 20) + 8 * M * k * (F + K), dtype=torch.uint8, device="cuda")
    else:
        M, N, K = case.get("M", 1), case["N"], case["K"]
        s["W"] = _weights(case["type"], N, K, gen)
        s["X"] = normal(M, K)
        s["bias"] = normal(N) * 0.5 if case["bias"] else None
        s["mul"] = normal(M, N) if case["mul"] else None
        s["residual"] = normal(M, N) if case["residual"] else None
        if op == "gemm":
            s["scratch"] = torch.zeros(GEMM_SCRATCH, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain form

def _f16(b):
    return b.contiguous().view(torch.float16)[..., 0].float()


def _dequant(raw, t, K):
    """f32 [..., K] of uint8 rows [..., row bytes]."""
    v, nbytes = BLOCKS[t]
    b = raw.unflatten(-1, (K // v, nbytes))
    if t in ("q4_K", "q5_K"):
        s = b[..., 4:16]
        sc = torch.cat([s[..., 0:4] & 63, (s[..., 8:12] & 15) | ((s[..., 0:4] >> 6) << 4)], -1)
        mn = torch.cat([s[..., 4:8] & 63, (s[..., 8:12] >> 4) | ((s[..., 4:8] >> 6) << 4)], -1)
        q = b[..., 16:144] if t == "q4_K" else b[..., 48:176]
        q = q.unflatten(-1, (4, 1, 32))
        codes = torch.cat([q & 15, q >> 4], -2).flatten(-3, -2)             # [8, 32]
        if t == "q5_K":
            bit = torch.arange(8, dtype=torch.uint8, device=raw.device).view(8, 1)
            codes = codes + (((b[..., None, 16:48] >> bit) & 1) << 4)
        scale = _f16(b[..., 0:2])[..., None] * sc.float()
        low = _f16(b[..., 2:4])[..., None] * mn.float()
        w = codes.float() * scale[..., None] - low[..., None]
    elif t == "q6_K":
        ql, qh = b[..., 0:128].unflatten(-1, (2, 2, 32)), b[..., 128:192].unflatten(-1, (2, 32))
        lo = torch.cat([ql & 15, ql >> 4], -2)                              # [2, 4, 32]
        two = torch.arange(0, 8, 2, dtype=torch.uint8, device=raw.device).view(4, 1)
        codes = (lo | (((qh[..., None, :] >> two) & 3) << 4)).float() - 32.0
        sc = b[..., 192:208].contiguous().view(torch.int8).float() * _f16(b[..., 208:210])[..., None]
        w = codes.reshape(*codes.shape[:-3], 16, 16) * sc[..., None]
    elif t == "q8_0":
        w = b[..., 2:34].contiguous().view(torch.int8).float() * _f16(b[..., 0:2])[..., None]
    else:
        five, has_min = t[1] == "5", t.endswith("_1")
        at = 4 if has_min else 2
        q = b[..., at + 4 * five:]
        codes = torch.cat([q & 15, q >> 4], -1)
        if five:
            bit = torch.arange(8, dtype=torch.uint8, device=raw.device)
            high = ((b[..., at:at + 4, None] >> bit) & 1).flatten(-2)
            codes = codes | (high << 4)
        d = _f16(b[..., 0:2])[..., None]
        if has_min:
            w = codes.float() * d + _f16(b[..., 2:4])[..., None]
        else:
            w = (codes.float() - (16.0 if five else 8.0)) * d
    return w.reshape(*raw.shape[:-1], K)


def _act(v, name):
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    if name == "gelu_erf":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    if name == "relu":
        return torch.clamp(v, min=0.0)
    return v


def _plain_route(s):
    c = s["case"]
    logits = s["X"].double() @ s["Wr"].double().t()    # in 64 bits: a choice next to a border has to fall the same way
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    if s["bias"] is not None:
        key = p + s["bias"].double()
    else:
        key = logits
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(p, 1, ids)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "wts": w.float()}


def _plain_moe(s):
    c = s["case"]
    M, K, F, E, k = (c[n] for n in ("M", "K", "F", "E", "k"))
    X, ids, wts = s["X"], s["ids"].long(), s["wts"]
    live = (ids >= 0) & (ids < E)
    wts = torch.where(live, wts, 0.0)
    ids = torch.where(live, ids, 0)
    if M * k < E:       # the chosen experts' weights, pair by pair
        p = ids.reshape(-1)
        x = X.repeat_interleave(k, 0).unsqueeze(-1)
        g = torch.matmul(_dequant(s["Wg"].view(E, F, -1)[p], c["gu"], K), x)
        u = torch.matmul(_dequant(s["Wu"].view(E, F, -1)[p], c["gu"], K), x)
        y = torch.matmul(_dequant(s["Wd"].view(E, K, -1)[p], c["down"], F), _act(g, c["act"]) * u)
        y = (y.view(M, k, K) * wts.unsqueeze(-1)).sum(1)
    else:               # every expert on every token, then the chosen ones' weighted sum
        xt = X.t().contiguous()
        g = _dequant(s["Wg"], c["gu"], K) @ xt
        u = _dequant(s["Wu"], c["gu"], K) @ xt
        h = (_act(g, c["act"]) * u).view(E, F, M)
        d = torch.matmul(_dequant(s["Wd"], c["down"], F).view(E, K, F), h)
        share = torch.zeros((E, M), device=X.device).index_put_(
            (ids, torch.arange(M, device=X.device).unsqueeze(1).expand(M, k)), wts, accumulate=True)
        y = (d * share.unsqueeze(1)).sum(0).t()
    return y + s["residual"] if s["residual"] is not None else y.contiguous()


def _epilogue(acc, s):
    v = acc if s["bias"] is None else acc + s["bias"]
    v = _act(v, s["case"]["act"])
    v = v if s["mul"] is None else v * s["mul"]
    return v if s["residual"] is None else v + s["residual"]


def _plain_gemm(s):
    c = s["case"]
    M, K = s["X"].shape
    x = s["X"].view(M, K // 32, 32)     # the product's activations: 8-bit codes of blocks of 32
    amax = x.abs().amax(-1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)
    codes = torch.where(scale > 0, torch.clamp(torch.round(x / torch.where(scale > 0, scale, 1.0)), -127, 127), 0.0)
    return _epilogue((codes * scale).view(M, K) @ _dequant(s["W"], c["type"], K).t(), s)


def _plain_gemv(s):
    c = s["case"]
    return _epilogue(s["X"] @ _dequant(s["W"], c["type"], c["K"]).t(), s)


# ------------------------------------------------------------------ the framework's calls

def _own(s):
    from block_quantized_matmul_mq_amd import mq
    c = s["case"]
    if "ready" not in s:
        mq.init(s["X"].device.index or 0)
        s["ready"] = True
    types = {"q4_0": mq.Q4_0, "q4_1": mq.Q4_1, "q5_0": mq.Q5_0, "q5_1": mq.Q5_1, "q8_0": mq.Q8_0, "q4_K": mq.Q4_K,
             "q5_K": mq.Q5_K, "q6_K": mq.Q6_K}
    acts = {"none": mq.ACT_NONE, "silu": mq.ACT_SILU, "gelu_tanh": mq.ACT_GELU_TANH, "gelu_erf": mq.ACT_GELU_ERF,
            "relu": mq.ACT_RELU}
    if c["op"] == "route":
        score = {"softmax": mq.SCORE_SOFTMAX, "sigmoid": mq.SCORE_SIGMOID}[c["score"]]
        ids, wts = mq.moe_route(s["X"], s["Wr"], c["k"], bias=s["bias"], score=score, norm=c["norm"],
                                scratch=s["scratch"])
        return {"ids": ids, "wts": wts}
    if c["op"] == "moe":
        return mq.moe_ffn(s["Wg"], s["Wu"], types[c["gu"]], s["Wd"], types[c["down"]], s["X"], s["ids"], s["wts"],
                          c["E"], c["F"], act=acts[c["act"]], residual=s["residual"], scratch=s["scratch"])
    ep = dict(bias=s["bias"], act=acts[c["act"]], mul=s["mul"], residual=s["residual"])
    if c["op"] == "gemv":
        return mq.gemv_ep(s["W"], types[c["type"]], s["X"], c["N"], c["K"], **ep).view(1, c["N"])
    Xq = mq.quantize_act(s["X"])
    return mq.gemm_ep(s["W"], types[c["type"]], Xq, c["M"], c["N"], c["K"], scratch=s["scratch"], **ep)


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "moe": _plain_moe, "gemv": _plain_gemv, "gemm": _plain_gemm}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits, from the definitions

def _tables(t):
    """Per value of a block: (byte, shift, mask) of the low bits and of the high bits (mask 0: none), the
    high bits' weight, the code offset, and for the K-quants the value's sub-block."""
    v = np.arange(BLOCKS[t][0])
    if t in ("q4_K", "q5_K"):
        base = 16 if t == "q4_K" else 48
        return ((base + 32 * (v // 64) + v % 32, 4 * (v // 32 % 2), 15),
                (16 + v % 32, v // 32, 1 if t == "q5_K" else 0), 16, 0, v // 32)
    if t == "q6_K":
        h, r, l = v // 128, v % 128 // 32, v % 32
        return ((64 * h + 32 * (r % 2) + l, 4 * (r // 2), 15), (128 + 32 * h + l, 2 * r, 3), 16, 32, v // 16)
    at = (4 if t.endswith("_1") else 2)
    five = t[1] == "5"
    return ((at + (4 if five else 0) + v % 16, 4 * (v // 16), 15), (at + v // 8, v % 8, 1 if five else 0), 16,
            (0 if t.endswith("_1") else 16 if five else 8), v * 0)


def _exact_weights(raw, t, K):
    v, nbytes = BLOCKS[t]
    b = raw.reshape(raw.shape[0], K // v, nbytes).int()

    def half(at):
        bits = b[..., at] + 256 * b[..., at + 1]
        frac, ex = (bits & 1023).double(), (bits >> 10) & 31
        mag = torch.where(ex == 0, frac * 2.0 ** -24,
                          (1024.0 + frac) * torch.pow(2.0, (ex - 25).double()))
        return torch.where(bits >= 32768, -mag, mag).unsqueeze(-1)

    def signed(x):
        return torch.where(x > 127, x - 256, x).double()

    if t == "q8_0":
        return (half(0) * signed(b[..., 2:34])).reshape(-1, K)

    def pick(field):
        at, shift, mask = field
        return (b[..., torch.as_tensor(at, device=b.device)] >> torch.as_tensor(shift, device=b.device)) & mask

    low, high, weight, offset, sub = _tables(t)
    codes = (pick(low) + weight * pick(high)).double() - offset if high[2] else pick(low).double() - offset
    if t in ("q4_K", "q5_K"):
        j = torch.as_tensor(sub, device=b.device)
        first, k = j < 4, j % 4
        s = b[..., 4:16]
        sc = torch.where(first, s[..., k] % 64, s[..., 8 + k] % 16 + 16 * (s[..., k] // 64)).double()
        mn = torch.where(first, s[..., 4 + k] % 64, s[..., 8 + k] // 16 + 16 * (s[..., 4 + k] // 64)).double()
        w = half(0) * sc * codes - half(2) * mn
    elif t == "q6_K":
        w = half(208) * signed(b[..., 192:208])[..., torch.as_tensor(sub, device=b.device)] * codes
    else:
        w = half(0) * codes + (half(2) if t.endswith("_1") else 0.0)
    return w.reshape(-1, K)


def _exact_act(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu_tanh":
        return v * torch.sigmoid(2.0 * np.sqrt(2.0 / np.pi) * (v + 0.044715 * v ** 3))
    if name == "gelu_erf":
        return v * 0.5 * torch.special.erfc(-v / np.sqrt(2.0))
    return torch.where(v > 0, v, 0.0) if name == "relu" else v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        X, W = s["X"].cpu().numpy().astype(np.float64), s["Wr"].cpu().numpy().astype(np.float64)
        z = X @ W.T
        p = np.exp(z - z.max(1, keepdims=True))
        p = p / p.sum(1, keepdims=True) if case["score"] == "softmax" else 1.0 / (1.0 + np.exp(-z))
        key = z if s["bias"] is None else p + s["bias"].cpu().numpy().astype(np.float64)
        ids = np.argsort(-key, axis=1, kind="stable")[:, :case["k"]]
        w = np.take_along_axis(p, ids, 1)
        return {"ids": ids.astype(np.int32), "wts": w / w.sum(1, keepdims=True) if case["norm"] else w}
    X = s["X"].double()
    if op == "moe":
        M, K, F, E = (case[n] for n in ("M", "K", "F", "E"))
        y = torch.zeros((M, K), dtype=torch.float64, device="cuda")
        ids = s["ids"].cpu().numpy()
        for e in range(E):
            m, j = (torch.as_tensor(i, device="cuda") for i in np.nonzero(ids == e))
            if m.numel():
                g = X[m] @ _exact_weights(s["Wg"][e * F:(e + 1) * F], case["gu"], K).t()
                u = X[m] @ _exact_weights(s["Wu"][e * F:(e + 1) * F], case["gu"], K).t()
                d = (_exact_act(g, case["act"]) * u) @ _exact_weights(s["Wd"][e * K:(e + 1) * K], case["down"], F).t()
                y.index_add_(0, m, d * s["wts"][m, j].double().unsqueeze(1))
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "gemm":    # what the product takes its activations for: round(x / (amax / 127)) of 32 values, in float32
        x = s["X"].cpu().numpy().reshape(-1, 32)
        scale = (np.abs(x).max(1, keepdims=True) / np.float32(127)).astype(np.float32)
        q = np.rint(np.divide(x, scale, out=np.zeros_like(x), where=scale > 0))
        X = torch.from_numpy(np.clip(q, -127, 127).astype(np.float64) * scale).cuda().view(X.shape)
    y = torch.cat([X @ _exact_weights(w, case["type"], case["K"]).t() for w in s["W"].split(4096)], 1)
    y = y if s["bias"] is None else y + s["bias"].double()
    y = _exact_act(y, case["act"])
    y = y if s["mul"] is None else y * s["mul"].double()
    return y if s["residual"] is None else y + s["residual"].double()
