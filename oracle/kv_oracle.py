"""Oracle of the operators on the paged cache and of sampling: numpy in f64, from the definitions in
include/mq.h, value by value where that is affordable.  Shares no code with the HIP path."""

import numpy as np

Q4_0, Q8_0 = 2, 8
BITS = {Q4_0: 4, Q8_0: 8}
OFFSET = {Q4_0: 8, Q8_0: 128}


def chunk_bytes(qtype, page, dim):
    return 2 * page * (dim * BITS[qtype] // 8 + dim // 16)


def places(qtype, page, dim):
    """(K byte, V byte, shift of K's code, shift of V's, K scale's byte, V scale's), int [page, dim] each, of every
    token and dimension in a page's chunk of one head."""
    bits, nb = BITS[qtype], dim // 32
    t, d = np.meshgrid(np.arange(page), np.arange(dim), indexing="ij")
    row = dim * bits // 8
    b, g, n = d // 32, d % 32 // 8, d % 8
    k_bit = 8 * (t * row) + 8 * ((g * nb + b) * bits) + n * bits
    run = 256 // bits
    i, j, c = d // run, d % run // 16, d % 16
    unit = ((t % 16) // 4 * 16 + c) * 2 + t % 4 // 2
    v_bit = 8 * (page * row + 16 * row * (t // 16) + 4 * (unit * (dim // run) + i) + 2 * (t % 2)) + j * bits
    ks = 2 * page * row + 2 * (t * nb + b)
    return k_bit // 8, v_bit // 8, k_bit % 8, v_bit % 8, ks, ks + 2 * page * nb


def half_bits(x):
    return np.asarray(x, dtype=np.float32).astype(np.float16).view(np.uint16)


def quantize(x, qtype):
    """(scale f16 bits [.., n/32], codes [.., n]) of f32 rows; codes as they are stored."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        if qtype == Q4_0:
            at = np.argmax(np.abs(b), -1)
            m = np.take_along_axis(b, at[..., None], -1)[..., 0]
            d = (m / np.float32(-8)).astype(np.float16)
        else:
            d = (np.abs(b).max(-1) / np.float32(127)).astype(np.float16)
        bad = ~np.isfinite(b).all(-1) | ~np.isfinite(d)
        d = np.where(bad, np.float16(np.nan), np.where(d == 0, np.float16(0), d))     # (never -0)
        df = d.astype(np.float32)[..., None]
        ok = (df != 0) & ~bad[..., None]
        r = np.rint(np.where(ok, b, 0) / np.where(ok, df, 1).astype(np.float32))
    code = np.clip(r + 8, 0, 15) if qtype == Q4_0 else np.clip(r, -127, 127) + 128
    code = np.where(ok, code, OFFSET[qtype]).astype(np.int64)
    return d.view(np.uint16), code.reshape(x.shape)


def values(scale_bits, codes, qtype):
    d = np.asarray(scale_bits, dtype=np.uint16).view(np.float16).astype(np.float64)
    c = codes.reshape(*codes.shape[:-1], -1, 32) - OFFSET[qtype]
    return (c * d[..., None]).reshape(codes.shape)


def normed(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    return x / np.sqrt(np.mean(x * x, -1, keepdims=True) + float(np.float32(eps))) * np.asarray(w, dtype=np.float64)


def rotated(x, pos, inv_freq, rope):
    """x f64 [T, heads, dim], pos [T]; rope 0, 1 (halves) or 2 (neighbours)."""
    if rope == 0:
        return x
    y = x.copy()
    half = len(inv_freq)
    for j in range(half):
        a = np.asarray(pos, dtype=np.float64) * float(inv_freq[j])
        p, q = (j, j + half) if rope == 1 else (2 * j, 2 * j + 1)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        y[:, :, p] = x[:, :, p] * c - x[:, :, q] * s
        y[:, :, q] = x[:, :, q] * c + x[:, :, p] * s
    return y


def rows_of(q_start, kv_len, T):
    """(sequence, position) of each row; sequence -1 for a row of no sequence."""
    out = []
    for t in range(T):
        b = [i for i in range(len(kv_len)) if q_start[i] <= t < q_start[i + 1]]
        out.append((b[0], int(kv_len[b[0]]) - (int(q_start[b[0] + 1]) - t)) if b else (-1, 0))
    return out


def place(table, pages, page, b, pos):
    """(page, slot) of a position, or None."""
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    p = int(table[b, pos // page])
    return (p, pos % page) if 0 <= p < pages else None


def put(data, qtype, page, heads, dim, p, slot, h, which, scale_bits, codes):
    """Writes one token's row of head h (which: 0 keys, 1 values) into the cache's bytes."""
    at = places(qtype, page, dim)
    chunk = data[(p * heads + h) * chunk_bytes(qtype, page, dim):][:chunk_bytes(qtype, page, dim)]
    mask = (1 << BITS[qtype]) - 1
    for d in range(dim):
        byte, shift = int(at[which][slot, d]), int(at[2 + which][slot, d])
        chunk[byte] = (int(chunk[byte]) & ~(mask << shift) & 255) | (int(codes[d]) << shift)
    for b in range(dim // 32):
        s = int(at[4 + which][slot, 32 * b])
        chunk[s], chunk[s + 1] = int(scale_bits[b]) & 255, int(scale_bits[b]) >> 8


def get(data, qtype, page, heads, dim):
    """(K, V) f64 [pages, heads, page, dim] of the whole cache."""
    at = places(qtype, page, dim)
    raw = data.reshape(-1, heads, chunk_bytes(qtype, page, dim)).astype(np.int64)
    mask = (1 << BITS[qtype]) - 1
    out = []
    for which in (0, 1):
        code = (raw[:, :, at[which]] >> at[2 + which]) & mask
        bits = (raw[:, :, at[4 + which]] | raw[:, :, at[4 + which] + 1] << 8).astype(np.uint16)
        out.append((code - OFFSET[qtype]) * bits.view(np.float16).astype(np.float64))
    return out


def attention(q, keys, vals, seen, scale):
    """f64 [heads, dim] of one row q [heads, dim] over keys, vals [kv heads, n, dim] where seen [n]."""
    G = q.shape[0] // keys.shape[0]
    out = np.zeros(q.shape)
    if not seen.any():
        return out
    for h in range(q.shape[0]):
        s = scale * (keys[h // G][seen] @ q[h].astype(np.float64))
        e = np.exp(s - s.max())
        out[h] = (e / e.sum()) @ vals[h // G][seen]
    return out


def attn(data, qtype, pages, page, heads, dim, q_start, kv_len, table, q, scale, causal=True, window=0):
    """f64 [T, q_heads, dim]; rows of no sequence NaN (they are not written)."""
    K, V = get(data, qtype, page, heads, dim)
    T = q.shape[0]
    out = np.full(q.shape, np.nan)
    for t, (b, pos) in enumerate(rows_of(q_start, kv_len, T)):
        if b < 0:
            continue
        n = max(0, int(kv_len[b]))
        spots = [place(table, pages, page, b, j) for j in range(n)]
        j = np.arange(n)
        seen = np.array([s is not None for s in spots], dtype=bool)
        if causal:
            seen &= j <= pos
            if window:
                seen &= j > pos - window
        at = [s or (0, 0) for s in spots]
        p, s = np.array([a[0] for a in at], dtype=int), np.array([a[1] for a in at], dtype=int)
        out[t] = attention(q[t], K[p, :, s].transpose(1, 0, 2), V[p, :, s].transpose(1, 0, 2), seen, scale)
    return out


def sample(logits, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(id, probability) of one row, walked token by token in falling order; a token whose e is under half of
    2^-43 is never the choice."""
    l = np.asarray(logits, dtype=np.float64)
    order = [i for i in np.argsort(-np.where(np.isnan(l), -np.inf, l), kind="stable") if l[i] > -np.inf]
    if not order:
        return -1, 0.0
    if not T > 0:
        return int(order[0]), 1.0
    top = l[order[0]]
    e = {i: 1.0 if l[i] == top else float(np.exp((l[i] - top) / T)) for i in order}
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        goal, have, kept = top_p * sum(e[i] for i in order), 0.0, []
        for i in order:
            if kept and have >= goal:
                break
            kept.append(i)
            have += e[i]
        order = kept
    order = [i for r, i in enumerate(order) if r == 0 or e[i] >= min(min_p, 1.0)]
    total = sum(e[i] for i in order)
    have = 0.0
    for i in sorted(order):
        have += e[i]
        if np.rint(e[i] * 2.0 ** 43) == 0:
            continue
        last = i
        if have > u * total:
            break
    return int(last), e[last] / total
