// mq_moe_ffn: a mixture-of-experts feed-forward layer for a few tokens,
//   Y[m] = residual[m] + sum_j w[m][j] * Wd_e ( act(Wg_e X[m]) * (Wu_e X[m]) ),   e = ids[m][j],
// over block-quantized expert weights and f32 activations.  (token, choice) pairs p = m k + j.
//
// What bounds it.  A few tokens touch each weight of a chosen expert only once or a few
// times, so the floor is the chosen experts' bytes from HBM; everything here is arranged to
// keep weight loads in flight and to spend few instructions per weight.
//
// Split.  Two launches, because every output of the down product needs every h of its token:
//   up    one workgroup per (expert, 16 TW rows of F): both the gate and the up rows, so that
//         act(g) * u is formed where both sums meet; h goes to scratch, f32 [pair][F].
//   down  few pairs: one workgroup per 16 rows of Y for all pairs, which sums the pairs itself
//         (nothing is exchanged between workgroups); many pairs: one per (expert, 16 TW rows),
//         weighted partial rows to scratch [pair][K], and a third launch adds each token's k
//         rows in choice order.
// With many pairs the workgroups of `up` and `down` collect the pairs of their expert, so that
// an expert's weights are read once for all its tokens (in chunks of at most 8).
//
// Arithmetic.  The exact-integer scheme of the GEMV kernels: per 32-value block of the
// activations x = 2^-s v with v an integer of at most 22 bits (relative to the block's largest
// value the staged x is off by at most 2^-22), v = 65536 d2 + 256 d1 + d0 in signed bytes.
// v_mfma_i32_16x16x64_i8 per 16-value chunk of four units at a time:
//   B (64 x 16): column n = weight row n of the tile, lane group q (lanes 16q .. 16q + 15)
//                holds 16 codes of unit q (64 of the 256 values of a group);
//   A (16 x 64): row 4q + p (p < 3) = digit plane p of the same 16 values in lane group q,
//                zero elsewhere,
// so lane (n, q) receives exactly its own unit's three plane sums (all exact) and applies its own
// block scales in f32.  The four units of a row are summed by lane swaps; each (group, tile,
// token) leaves one partial per row in LDS, and the partials of a row are summed in a fixed
// order: the result does not depend on timing.
//
// A lane's 64 values of a weight row are loaded straight into registers (16-byte loads, also
// where the block starts on a 2-byte boundary), several items ahead.  Items are ordered group
// first, so a wave keeps the tokens' A operands in registers while it walks the tiles.
#include <algorithm>
#include <type_traits>

#include "mq_device.h"
#include "mq_epilogue.h"
#include "mq_internal.h"
#include "weight_units.h"

namespace mq {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kFracBits = 22;
constexpr int kTokens = 8;                  // tokens of one expert computed together
constexpr int kUnitBytes = 768 + 32 + 64;   // staged 256 values: digit planes, block scales, sums
constexpr int kStageBudget = 72 * 1024;     // LDS of staged activations and partials: two workgroups per CU

__device__ __forceinline__ uint4 load16(const uint8_t* p) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);   // (unaligned: one 16-byte load)
    return v;
}
__device__ __forceinline__ uint32_t load4(const uint8_t* p) {
    uint32_t v;
    __builtin_memcpy(&v, p, 4);
    return v;
}

// LDS writes of every wave visible, without waiting for loads in flight
// (__syncthreads waits for those too).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

__device__ __forceinline__ v4i as_v4i(const uint4 v) { return v4i{int(v.x), int(v.y), int(v.z), int(v.w)}; }

// ------------------------------------------------------------------ weights
// Scales per lane unit (64 values): one per 32-value block, or per 16-value run (Q6_K).
template <int QT> constexpr int scales_per_unit() { return QT == kQ6_K ? 4 : 2; }
// A code is unsigned with an offset taken off through the integer sum of v (Q6_K, Q4_0, Q5_0)
template <int QT> constexpr int code_offset() { return QT == kQ6_K ? 32 : QT == kQ4_0 ? 8 : QT == kQ5_0 ? 16 : 0; }
// Whether |sum code v| can pass 2^31 (the plane sums are then combined in f32): 5-bit codes
// without an offset and 8-bit codes.  (The others: 32 * 15 * 2^22 < 2^31; with the offset taken
// off, modulo 2^32, 16 * 32 * (2^22 - 1) and 32 * 16 * (2^22 - 1) < 2^31.)
template <int QT> constexpr bool wide_sums() { return QT == kQ8_0 || QT == kQ5_K || QT == kQ5_1; }

// One item for one lane: unit q (64 values) of 256-value group g of one weight row, decoded
// to four chunks of 16 codes (MFMA B operands), the scales of its blocks and their minima
// (value = ds * code - dm).
template <int QT>
struct Decoded {
    v4i chunk[4];
    float ds[scales_per_unit<QT>()];
    float dm[2];
};

template <int QT>
struct Bytes;

template <>
struct Bytes<kQ4_K> {
    uint4 hd, c0, c1;
    __device__ void load(const uint8_t* row, int g, int q, int, int, int) {
        const uint8_t* b = row + 144 * g;
        hd = load16(b);
        c0 = load16(b + 16 + 32 * q);
        c1 = load16(b + 32 + 32 * q);
    }
    __device__ void decode(Decoded<kQ4_K>& o, int q) const {
        const v4i a = as_v4i(c0), b = as_v4i(c1);
        o.chunk[0] = a & 0x0F0F0F0F;
        o.chunk[1] = b & 0x0F0F0F0F;
        o.chunk[2] = (a >> 4) & 0x0F0F0F0F;
        o.chunk[3] = (b >> 4) & 0x0F0F0F0F;
        RawQ4K r;
        r.hd = hd;
        uint32_t sc, mn;
        r.scale_min(q, sc, mn);
        const float d = r.d(), dmin = r.dmin();   // (f16 times 6 bits: exact products)
        o.ds[0] = d * ubyte_f<0>(sc);
        o.ds[1] = d * ubyte_f<1>(sc);
        o.dm[0] = dmin * ubyte_f<0>(mn);
        o.dm[1] = dmin * ubyte_f<1>(mn);
    }
};

template <>
struct Bytes<kQ5_K> {
    uint4 hd, h0, h1, c0, c1;
    __device__ void load(const uint8_t* row, int g, int q, int, int, int) {
        const uint8_t* b = row + 176 * g;
        hd = load16(b);
        h0 = load16(b + 16);
        h1 = load16(b + 32);
        c0 = load16(b + 48 + 32 * q);
        c1 = load16(b + 64 + 32 * q);
    }
    __device__ void decode(Decoded<kQ5_K>& o, int q) const {
        const v4i a = as_v4i(c0), b = as_v4i(c1);
        const v4i ha = as_v4i(h0) >> (2 * q), hb = as_v4i(h1) >> (2 * q);
        o.chunk[0] = (a & 0x0F0F0F0F) | ((ha & 0x01010101) << 4);
        o.chunk[1] = (b & 0x0F0F0F0F) | ((hb & 0x01010101) << 4);
        o.chunk[2] = ((a >> 4) & 0x0F0F0F0F) | (((ha >> 1) & 0x01010101) << 4);
        o.chunk[3] = ((b >> 4) & 0x0F0F0F0F) | (((hb >> 1) & 0x01010101) << 4);
        RawQ5K r;
        r.hd = hd;
        uint32_t sc, mn;
        r.scale_min(q, sc, mn);
        const float d = r.d(), dmin = r.dmin();
        o.ds[0] = d * ubyte_f<0>(sc);
        o.ds[1] = d * ubyte_f<1>(sc);
        o.dm[0] = dmin * ubyte_f<0>(mn);
        o.dm[1] = dmin * ubyte_f<1>(mn);
    }
};

// Unit q of Q6_K: super-block half h = q / 2, lanes l0 = 16 (q % 2) .. + 15 of each of the four
// 32-value runs of that half; chunk c = run c (one sub-scale each).
template <>
struct Bytes<kQ6_K> {
    uint4 a, b, hq;
    uint32_t s0, s1, dbits;
    __device__ void load(const uint8_t* row, int g, int q, int, int stride, int off) {
        const uint8_t* blk = row + stride * g + off;
        const int h = q >> 1, l0 = 16 * (q & 1);
        a = load16(blk + 64 * h + l0);
        b = load16(blk + 64 * h + 32 + l0);
        hq = load16(blk + 128 + 32 * h + l0);
        s0 = load4(blk + 192 + 8 * h);
        s1 = load4(blk + 196 + 8 * h);
        dbits = load_u16(blk + 208);
    }
    __device__ void decode(Decoded<kQ6_K>& o, int q) const {
        const v4i A = as_v4i(a), B = as_v4i(b), H = as_v4i(hq);
        const float d = half_bits_to_float(dbits);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const v4i src = (c & 1) ? B : A;
            o.chunk[c] = ((c < 2 ? src : (src >> 4)) & 0x0F0F0F0F) | (((H >> (2 * c)) & 0x03030303) << 4);
            o.ds[c] = d * RawQ6K::subscale(c, q, s0, s1);   // (f16 times 8 bits: exact)
        }
        o.dm[0] = o.dm[1] = 0.f;
    }
};

// The 32-value types: unit q = blocks 2q and 2q + 1 of the group's eight.  In a last group of
// fewer than eight blocks the lanes past the row's end read its last block again (their staged
// activations are zero).
template <>
struct Bytes<kQ8_0> {
    uint4 c[4];
    uint32_t db[2];
    __device__ void load(const uint8_t* row, int g, int q, int blocks, int stride, int off) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* b = row + stride * min(8 * g + 2 * q + i, blocks - 1) + off;
            db[i] = load_u16(b);
            c[2 * i] = load16(b + 2);
            c[2 * i + 1] = load16(b + 18);
        }
    }
    __device__ void decode(Decoded<kQ8_0>& o, int) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) o.chunk[k] = as_v4i(c[k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o.ds[i] = half_bits_to_float(db[i]);
            o.dm[i] = 0.f;
        }
    }
};

template <int QT>
struct LegacyBytes {
    using L = Legacy<QT>;
    uint4 c[2];
    uint32_t db[2], hb[2];
    __device__ void load(const uint8_t* row, int g, int q, int blocks, int, int) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* b = row + L::kBytes * min(8 * g + 2 * q + i, blocks - 1);
            constexpr int at = L::kMin ? 4 : 2;
            db[i] = L::kMin ? load4(b) : load_u16(b);
            hb[i] = L::kHigh ? load4(b + at) : 0u;
            c[i] = load16(b + at + (L::kHigh ? 4 : 0));
        }
    }
    __device__ void decode(Decoded<QT>& o, int) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const v4i v = as_v4i(c[i]);
            v4i lo = v & 0x0F0F0F0F, hi = (v >> 4) & 0x0F0F0F0F;
            if constexpr (L::kHigh) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lo[k] |= int(spread4((hb[i] >> (4 * k)) & 15u) << 4);
                    hi[k] |= int(spread4((hb[i] >> (16 + 4 * k)) & 15u) << 4);
                }
            }
            o.chunk[2 * i] = lo;
            o.chunk[2 * i + 1] = hi;
            o.ds[i] = half_bits_to_float(db[i] & 0xFFFFu);
            o.dm[i] = L::kMin ? -half_bits_to_float(db[i] >> 16) : 0.f;
        }
    }
};
template <> struct Bytes<kQ4_0> : LegacyBytes<kQ4_0> {};
template <> struct Bytes<kQ4_1> : LegacyBytes<kQ4_1> {};
template <> struct Bytes<kQ5_0> : LegacyBytes<kQ5_0> {};
template <> struct Bytes<kQ5_1> : LegacyBytes<kQ5_1> {};

// ------------------------------------------------------------------ staged activations
// One unit of staged LDS: 256 values of one token (kUnitBytes): digit planes int8 [3][256],
// f32 scale 2^-s of each 32-value block, and what the type needs of the integer sums of v:
//   types with a minimum: f32 2^-s sum(v) per block; Q4_0, Q5_0: int32 sum(v) per block;
//   Q6_K: int32 sum(v) per 16-value run, run 2c + i of half h at 8 h + 4 i + c.
// All of them come from the same rounded v that the digits hold, so a code's offset or a
// minimum multiplies exactly the x that the codes meet.  A block that holds an infinity or a
// NaN has a NaN scale: every output of that token becomes NaN.
__device__ __forceinline__ uint32_t digits3(int v) { return (uint32_t(v) + 0x00808080u) ^ 0x00808080u; }

// Stage 256 values: lane l holds values 4l .. 4l + 3 (zeros past the row's end).
template <int QT>
__device__ __forceinline__ void stage_unit(uint8_t* unit, const float4 x, int lane) {
    float a = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
    a = lanes8_max(a);
    // v in (-2^22, 2^22): amax = m 2^E, m in [0.5, 1), s = 22 - E (at most 120: blocks below
    // 2^-98 keep fewer bits, an absolute error of 2^-121)
    const int s = min(kFracBits - __builtin_amdgcn_frexp_expf(a), 120);
    constexpr float kTop = 4194303.0f;
    auto integer = [&](float f) { return int(rintf(fminf(fmaxf(ldexpf(f, s), -kTop), kTop))); };
    const int v0 = integer(x.x), v1 = integer(x.y), v2 = integer(x.z), v3 = integer(x.w);
    const uint32_t r0 = digits3(v0), r1 = digits3(v1), r2 = digits3(v2), r3 = digits3(v3);
    const uint32_t t01 = __builtin_amdgcn_perm(r1, r0, 0x05010400u), t23 = __builtin_amdgcn_perm(r3, r2, 0x05010400u);
    const uint32_t u01 = __builtin_amdgcn_perm(r1, r0, 0x00000602u), u23 = __builtin_amdgcn_perm(r3, r2, 0x00000602u);
    uint32_t* planes = reinterpret_cast<uint32_t*>(unit);
    planes[lane] = __builtin_amdgcn_perm(t23, t01, 0x05040100u);
    planes[64 + lane] = __builtin_amdgcn_perm(t23, t01, 0x07060302u);
    planes[128 + lane] = __builtin_amdgcn_perm(u23, u01, 0x05040100u);
    float* scl = reinterpret_cast<float*>(unit + 768);
    // (0 * x is NaN for an infinity or a NaN and 0 otherwise; a sum keeps the NaN)
    float bad = 0.f * x.x + 0.f * x.y + (0.f * x.z + 0.f * x.w);
    bad = lanes8_sum(bad);
    const float scale = ldexpf(1.0f, -s) + bad;
    const int b = lane >> 3;
    if ((lane & 7) == 0) scl[b] = scale;
    int sum = (v0 + v1) + (v2 + v3);
    if constexpr (QT == kQ6_K) {
        sum = lanes8_sum<2>(sum);   // 16-value runs: run 2 b + i, b = 4 h + c
        if ((lane & 3) == 0)
            reinterpret_cast<int*>(unit + 800)[8 * (b >> 2) + 4 * ((lane >> 2) & 1) + (b & 3)] = sum;
    } else if constexpr (code_offset<QT>() != 0) {
        sum = lanes8_sum(sum);
        if ((lane & 7) == 0) reinterpret_cast<int*>(unit + 800)[b] = sum;
    } else if constexpr (has_min_term<QT>()) {
        sum = lanes8_sum(sum);
        if ((lane & 7) == 0) reinterpret_cast<float*>(unit + 800)[b] = float(sum) * scale;
    }
}

// ------------------------------------------------------------------ products
// Sum over the lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float sum_units(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    const float s = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// The A operands of T tokens' staged units (consecutive in LDS) for this lane.
template <int QT, int T>
struct Operands {
    v4i a[T][4];
    __device__ void load(const uint8_t* lds, int lane_off, int unit0, bool live, const uint8_t* zero) {
        constexpr int step = QT == kQ6_K ? 32 : 16;   // bytes between a lane's chunks
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint8_t* p = live ? lds + (unit0 + t) * kUnitBytes + lane_off : zero;
#pragma unroll
            for (int c = 0; c < 4; ++c) a[t][c] = *reinterpret_cast<const v4i*>(p + step * c);
        }
    }
};

// This lane's unit of one item against one token: its share of the row's dot product.
template <int QT>
__device__ __forceinline__ float unit_dot(const Decoded<QT>& w, const v4i (&a)[4], const uint8_t* unit, int q) {
    constexpr int NS = scales_per_unit<QT>();
    const v4i z = {0, 0, 0, 0};
    float r = 0.f;
    float sc[NS];
    int si[NS];
    float sx[2];
    if constexpr (NS == 4) {
        const float4 f = *reinterpret_cast<const float4*>(unit + 768 + 16 * (q >> 1));
        sc[0] = f.x; sc[1] = f.y; sc[2] = f.z; sc[3] = f.w;
        const int4 i = *reinterpret_cast<const int4*>(unit + 800 + 32 * (q >> 1) + 16 * (q & 1));
        si[0] = i.x; si[1] = i.y; si[2] = i.z; si[3] = i.w;
    } else {
        const float2 f = *reinterpret_cast<const float2*>(unit + 768 + 8 * q);
        sc[0] = f.x; sc[1] = f.y;
        if constexpr (code_offset<QT>() != 0) {
            const int2 i = *reinterpret_cast<const int2*>(unit + 800 + 8 * q);
            si[0] = i.x; si[1] = i.y;
        }
        if constexpr (has_min_term<QT>()) {
            const float2 m = *reinterpret_cast<const float2*>(unit + 800 + 8 * q);
            sx[0] = m.x; sx[1] = m.y;
        }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        v4i c = z;
#pragma unroll
        for (int k = 0; k < 4 / NS; ++k)
            c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[s * (4 / NS) + k], w.chunk[s * (4 / NS) + k], c, 0, 0, 0);
        float f;
        if constexpr (wide_sums<QT>()) {
            f = fmaf(float(c[2]), 65536.0f, fmaf(float(c[1]), 256.0f, float(c[0])));
        } else {
            int i = int((((uint32_t(c[2]) << 8) + uint32_t(c[1])) << 8) + uint32_t(c[0]));
            if constexpr (code_offset<QT>() != 0) i = int(uint32_t(i) - uint32_t(code_offset<QT>()) * uint32_t(si[s]));
            f = float(i);
        }
        r = fmaf(w.ds[s] * sc[s], f, r);
    }
    if constexpr (has_min_term<QT>()) r = fmaf(-w.dm[0], sx[0], fmaf(-w.dm[1], sx[1], r));
    return r;
}

// Where an item of a wave is: where(i).  Its partials go to part[i T + t][16].
struct ItemAt {
    const uint8_t* row;   // the lane's weight row (block 0)
    int group;            // 256-value group of the row
    int unit;             // first of the T staged units
};

template <int QT, int T, int DEPTH, class Where>
__device__ __forceinline__ void prime_items(Bytes<QT> (&buf)[DEPTH], const Where& where, int i0, int i1, int q,
                                            int blocks, int stride, int off) {
#pragma unroll
    for (int j = 0; j < DEPTH; ++j)
        if (i0 + j < i1) {
            const ItemAt at = where(i0 + j);
            buf[j].load(at.row, at.group, q, blocks, stride, off);
        }
}

template <int QT, int T, int DEPTH, class Where>
__device__ __forceinline__ void run_items(Bytes<QT> (&buf)[DEPTH], const Where& where, int i0, int i1, int lane,
                                          const uint8_t* staged, const uint8_t* zero, float* part, int blocks,
                                          int stride, int off) {
    const int n = lane & 15, q = lane >> 4;
    const bool live = (n >> 2) == q && (n & 3) < 3;
    const int lane_off = 256 * (n & 3) + (QT == kQ6_K ? 128 * (q >> 1) + 16 * (q & 1) : 64 * q);
    Operands<QT, T> op;
    int have = -1;
    auto compute = [&](const Bytes<QT>& b, int i) {
        const ItemAt at = where(i);
        if (at.unit != have) {   // uniform
            op.load(staged, lane_off, at.unit, live, zero);
            have = at.unit;
        }
        Decoded<QT> w;
        b.decode(w, q);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float r = sum_units(unit_dot<QT>(w, op.a[t], staged + (at.unit + t) * kUnitBytes, q));
            if (q == 0) part[(i * T + t) * 16 + n] = r;
        }
    };
    auto load = [&](Bytes<QT>& b, int i) {
        const ItemAt at = where(i);
        b.load(at.row, at.group, q, blocks, stride, off);
    };
    int i = i0;
    // steady part: one load per computed item, no conditions (the compiler then waits for
    // exactly the item it needs); the drain issues no loads past the end
    for (; i + 2 * DEPTH <= i1; i += DEPTH) {
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) {
            compute(buf[j], i + j);
            load(buf[j], i + j + DEPTH);
        }
    }
#pragma unroll
    for (int j = 0; j < 2 * DEPTH; ++j) {
        if (i + j < i1) {
            compute(buf[j % DEPTH], i + j);
            if (j < DEPTH && i + j + DEPTH < i1) load(buf[j % DEPTH], i + j + DEPTH);
        }
    }
}

// The x of a wave's share of the units to stage, requested before the weights (a wave's loads
// return in order), staged after.  Units wave, wave + kWaves, ... of `units`.
constexpr int kEarly = 4;
struct EarlyX {
    float4 v[kEarly];
};
template <class Source>
__device__ __forceinline__ float4 unit_x(const Source& src, int u, int lane) {
    const float* p;
    int left;   // values from the unit's first to the row's end
    src(u, p, left);
    float4 v = {0.f, 0.f, 0.f, 0.f};
    if (4 * lane < left) v = reinterpret_cast<const float4*>(p)[lane];
    return v;
}
template <class Source>
__device__ __forceinline__ void early_x(EarlyX& e, const Source& src, int units, int wave, int lane) {
#pragma unroll
    for (int j = 0; j < kEarly; ++j) {
        const int u = wave + kWaves * j;
        if (u < units) e.v[j] = unit_x(src, u, lane);
    }
}
template <int QT, class Source>
__device__ __forceinline__ void stage_units(const EarlyX& e, const Source& src, uint8_t* staged, int units, int wave,
                                            int lane) {
#pragma unroll
    for (int j = 0; j < kEarly; ++j) {
        const int u = wave + kWaves * j;
        if (u < units) stage_unit<QT>(staged + u * kUnitBytes, e.v[j], lane);
    }
    for (int u = wave + kWaves * kEarly; u < units; u += kWaves)
        stage_unit<QT>(staged + u * kUnitBytes, unit_x(src, u, lane), lane);
}

struct MoeArgs {
    const uint8_t* w0;     // up: gate weights; down: down weights
    const uint8_t* w1;     // up: up weights
    const float* x;        // up: X [M][in]; down: h [pair][in]
    const int32_t* ids;    // [pairs]
    const float* wts;      // [pairs] (down)
    const float* residual; // [M][rows] or null (down, few pairs)
    float* out;            // up: h [pair][rows]; down: Y [M][rows], or weighted rows [pair][rows]
    int pairs, topk, experts;
    int in, rows;          // values per weight row, weight rows per expert
    int groups;            // 256-value groups per row
    int phase;             // groups staged at a time (few pairs' down: units)
    int tiles;             // 16-row tiles per workgroup
    int act;
    int stride, off;       // weight block layout
    int64_t row_bytes;
};

// The sum of one output's partials over its units u (groups of a row, or groups of a token's
// pairs): four running sums, of the u that leave 0, 1, 2, 3 modulo 4, kept over all phases and
// added as (0 + 1) + (2 + 3) at the end.  So the order is the same whether four threads hold one
// of them each (few outputs) or one thread all four, and wherever a phase ends: a token's bits do
// not depend on what else the workgroup computes.
struct RowSums {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    // `read(u)` is unit u's partial of this thread's output, u0 <= u < u1
    template <class Read>
    __device__ void add(bool split, int j, int u0, int u1, const Read& read) {
        if (split) {
            for (int u = u0 + ((j - u0) & 3); u < u1; u += 4) s[0] += read(u);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                for (int u = u0 + ((k - u0) & 3); u < u1; u += 4) s[k] += read(u);
        }
    }
    // the total, in the output's first thread; red[4][outputs] (LDS) is free before and after
    __device__ float total(bool split, int outputs, float* red) const {
        if (!split) return (s[0] + s[1]) + (s[2] + s[3]);
        const int tid = threadIdx.x;
        if (tid < 4 * outputs) red[tid] = s[0];
        lds_barrier();
        float v = 0.f;
        if (tid < outputs) v = (red[tid] + red[outputs + tid]) + (red[2 * outputs + tid] + red[3 * outputs + tid]);
        lds_barrier();
        return v;
    }
};

// ------------------------------------------------------------------ up, and down with many pairs
// blockIdx.x: 16 TW rows of the expert; blockIdx.y: slot.  PAIRS: the slot is a pair; else it is
// the slot-th chosen expert, and the workgroup takes all its pairs, kTokens at a time.
// LDS: pair list | staged units | partials | sums.
template <int QT, bool UP>
struct GroupShape {
    static constexpr int kMats = UP ? 2 : 1;
};

template <int QT, bool UP, int T, int DEPTH>
__device__ __forceinline__ void group_chunk(const MoeArgs& a, int expert, int tile0, int tiles, const int* list,
                                            int count, uint8_t* staged, const uint8_t* zero, float* part, float* red) {
    constexpr int kMats = GroupShape<QT, UP>::kMats;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q = lane >> 4;
    const int nt = tiles * kMats;
    const int blocks = QT == kQ4_K || QT == kQ5_K || QT == kQ6_K ? a.in >> 8 : a.in >> 5;
    const int64_t row0 = (int64_t(expert) * a.rows + 16 * tile0 + n) * a.row_bytes;
    // outputs o = (tile, token, row), of thread o, or of threads o, outputs + o, ... (RowSums)
    const int outputs = tiles * 16 * T;
    const bool split = 4 * outputs <= kThreads;
    const int j = split ? tid / outputs : 0, o = tid - j * outputs;
    const int o_tile = o / (16 * T), o_t = (o >> 4) & (T - 1), o_r = o & 15;
    const bool has_output = split ? j < 4 : tid < outputs;
    RowSums sums[kMats];
    for (int g0 = 0; g0 < a.groups; g0 += a.phase) {
        const int ng = min(a.phase, a.groups - g0);
        const int items = ng * nt;
        const int i0 = wave * items / kWaves, i1 = (wave + 1) * items / kWaves;
        auto where = [&](int i) {   // group-major: tiles (and both matrices) of one group in turn
            const int g = i / nt, m = i - g * nt;
            const int tile = UP ? m >> 1 : m;
            const uint8_t* w = UP && (m & 1) ? a.w1 : a.w0;
            return ItemAt{w + row0 + int64_t(16 * tile) * a.row_bytes, g0 + g, g * T};
        };
        auto source = [&](int u, const float*& p, int& left) {   // unit u = (group, token)
            const int g = u / T, t = u - g * T;
            const int pair = list[min(t, count - 1)];
            const int r = UP ? pair / a.topk : pair;
            p = a.x + int64_t(r) * a.in + 256 * (g0 + g);
            left = a.in - 256 * (g0 + g);
        };
        EarlyX ex;
        early_x(ex, source, ng * T, wave, lane);
        Bytes<QT> buf[DEPTH];
        prime_items<QT, T, DEPTH>(buf, where, i0, i1, q, blocks, a.stride, a.off);
        stage_units<QT>(ex, source, staged, ng * T, wave, lane);
        lds_barrier();
        run_items<QT, T, DEPTH>(buf, where, i0, i1, lane, staged, zero, part, blocks, a.stride, a.off);
        lds_barrier();
        if (has_output) {
#pragma unroll
            for (int mat = 0; mat < kMats; ++mat)
                sums[mat].add(split, j, g0, g0 + ng, [&](int g) {
                    return part[(((g - g0) * nt + o_tile * kMats + mat) * T + o_t) * 16 + o_r];
                });
        }
        lds_barrier();   // the partials and staged units are free
    }
    float v[kMats];
#pragma unroll
    for (int mat = 0; mat < kMats; ++mat) v[mat] = sums[mat].total(split, outputs, red);
    if (tid < outputs && o_t < count) {
        const int pair = list[o_t];
        float r;
        if constexpr (UP) r = activate(v[0], a.act) * v[1];
        else r = a.wts[pair] * v[0];
        a.out[int64_t(pair) * a.rows + 16 * (tile0 + o_tile) + o_r] = r;
    }
}

template <int QT, bool UP, bool PAIRS>
__global__ __launch_bounds__(kThreads, PAIRS ? 4 : 2) void moe_group_kernel(MoeArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t* zero = smem;                                     // 128 zero bytes
    unsigned* bits = reinterpret_cast<unsigned*>(smem + 128); // chosen experts, a bit each
    int* count_lds = reinterpret_cast<int*>(smem + 128 + kMoeMaxExperts / 8);
    float* red = reinterpret_cast<float*>(smem + 128 + kMoeMaxExperts / 8 + 16);
    int* list = reinterpret_cast<int*>(red + kThreads);
    const int list_room = PAIRS ? 4 : (a.pairs + 3) & ~3;
    uint8_t* staged = reinterpret_cast<uint8_t*>(list + list_room);
    const int tid = threadIdx.x;
    const int tile0 = blockIdx.x * a.tiles;
    const int tiles = min(a.tiles, a.rows / 16 - tile0);
    if (tid < 32) reinterpret_cast<unsigned*>(zero)[tid] = 0u;
    if constexpr (PAIRS) {
        const int pair = blockIdx.y;
        const int expert = a.ids[pair];
        if (unsigned(expert) >= unsigned(a.experts)) return;   // (uniform) not this layer's: adds nothing
        if (tid == 0) list[0] = pair;
        lds_barrier();
        float* part = reinterpret_cast<float*>(staged + a.phase * kUnitBytes);
        group_chunk<QT, UP, 1, 4>(a, expert, tile0, tiles, list, 1, staged, zero, part, red);
    } else {
        const int words = (a.experts + 31) >> 5;
        if (tid < words) bits[tid] = 0u;
        lds_barrier();
        for (int p = tid; p < a.pairs; p += kThreads) {
            const int e = a.ids[p];
            if (unsigned(e) < unsigned(a.experts)) atomicOr(&bits[e >> 5], 1u << (e & 31));
        }
        lds_barrier();
        int slot = blockIdx.y, expert = -1;   // the slot-th set bit
        for (int w = 0; w < words; ++w) {
            unsigned b = bits[w];
            const int c = __popc(b);
            if (slot < c) {
                for (; slot > 0; --slot) b &= b - 1;
                expert = 32 * w + __ffs(int(b)) - 1;
                break;
            }
            slot -= c;
        }
        if (expert < 0) return;   // (uniform) fewer chosen experts than slots
        if (tid < 64) {           // the expert's pairs, in order
            int n = 0;
            for (int p0 = 0; p0 < a.pairs; p0 += 64) {
                const int p = p0 + tid;
                const bool mine = p < a.pairs && a.ids[p] == expert;
                const unsigned long long m = __ballot(mine);
                if (mine) list[n + __popcll(m & ((1ull << tid) - 1))] = p;
                n += __popcll(m);
            }
            if (tid == 0) *count_lds = n;
        }
        lds_barrier();
        const int count = *count_lds;
        for (int c0 = 0; c0 < count; c0 += kTokens) {
            const int c = min(kTokens, count - c0);
            const int* l = list + c0;
            auto go = [&](auto t_c, auto depth_c) {
                constexpr int T = decltype(t_c)::value;
                float* part = reinterpret_cast<float*>(staged + a.phase * T * kUnitBytes);
                group_chunk<QT, UP, T, decltype(depth_c)::value>(a, expert, tile0, tiles, l, c, staged, zero, part,
                                                                 red);
            };
            if (c == 1) go(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
            else if (c == 2) go(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{});
            else if (c <= 4) go(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
            else go(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
            lds_barrier();
        }
    }
}

// ------------------------------------------------------------------ down with few pairs
// blockIdx.x: `tiles` 16-row tiles of Y, for every pair.  A unit is one 256-value group of one
// pair's h; an item is a unit with one tile.
template <int QT>
__global__ __launch_bounds__(kThreads, 4) void moe_down_pairs_kernel(MoeArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint8_t* zero = smem;
    int* count_lds = reinterpret_cast<int*>(smem + 128);
    float* red = reinterpret_cast<float*>(smem + 128 + 16);
    int* list = reinterpret_cast<int*>(red + kThreads);          // valid pairs
    int* expert_of = list + kMoeFewPairs;
    float* weight_of = reinterpret_cast<float*>(expert_of + kMoeFewPairs);
    int* first_of = reinterpret_cast<int*>(weight_of + kMoeFewPairs);   // valid pairs before token m's; [tokens + 1]
    uint8_t* staged = reinterpret_cast<uint8_t*>(first_of + kMoeFewPairs + 4);
    float* part = reinterpret_cast<float*>(staged + a.phase * kUnitBytes);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q = lane >> 4;
    if (tid < 32) reinterpret_cast<unsigned*>(zero)[tid] = 0u;
    if (tid < 64) {   // (kMoeFewPairs <= 64)
        const int e = tid < a.pairs ? a.ids[tid] : -1;
        const bool ok = unsigned(e) < unsigned(a.experts);
        const unsigned long long m = __ballot(ok);
        if (ok) {
            const int at = __popcll(m & ((1ull << tid) - 1));
            list[at] = tid;
            expert_of[at] = e;
            weight_of[at] = a.wts[tid];
        }
        if (tid == 0) *count_lds = __popcll(m);
        if (tid <= a.pairs / a.topk) {   // (kMoeFewPairs < 64: no shift by 64)
            const int before = tid * a.topk;
            first_of[tid] = __popcll(m & ((1ull << before) - 1));
        }
    }
    lds_barrier();
    const int valid = *count_lds;
    const int tile0 = blockIdx.x * a.tiles;
    const int nt = min(a.tiles, a.rows / 16 - tile0);
    const int blocks = QT == kQ4_K || QT == kQ5_K || QT == kQ6_K ? a.in >> 8 : a.in >> 5;
    const int tokens = a.pairs / a.topk;
    // outputs o = (tile, token, row)
    const int outputs = nt * 16 * tokens;     // (at most kThreads)
    const int units = valid * a.groups;
    const bool split = 4 * outputs <= kThreads;
    const int j = split ? tid / outputs : 0, o = tid - j * outputs;
    const int o_tile = o / (16 * tokens), o_m = (o >> 4) - o_tile * tokens, o_r = o & 15;
    const bool has_output = split ? j < 4 : tid < outputs;
    const int my0 = has_output ? first_of[o_m] * a.groups : 0;            // its token's units
    const int my1 = has_output ? first_of[o_m + 1] * a.groups : 0;
    RowSums sums;
    for (int u0 = 0; u0 < units; u0 += a.phase) {
        const int nu = min(a.phase, units - u0);
        const int items = nu * nt;
        const int i0 = wave * items / kWaves, i1 = (wave + 1) * items / kWaves;
        auto where = [&](int i) {
            const int u = i / nt, tile = i - u * nt;
            const int v = (u0 + u) / a.groups, g = (u0 + u) - v * a.groups;
            const int64_t row = int64_t(expert_of[v]) * a.rows + 16 * (tile0 + tile) + n;
            return ItemAt{a.w0 + row * a.row_bytes, g, u};
        };
        auto source = [&](int u, const float*& p, int& left) {
            const int v = (u0 + u) / a.groups, g = (u0 + u) - v * a.groups;
            p = a.x + int64_t(list[v]) * a.in + 256 * g;
            left = a.in - 256 * g;
        };
        EarlyX ex;
        early_x(ex, source, nu, wave, lane);
        Bytes<QT> buf[4];
        prime_items<QT, 1, 4>(buf, where, i0, i1, q, blocks, a.stride, a.off);
        stage_units<QT>(ex, source, staged, nu, wave, lane);
        lds_barrier();
        run_items<QT, 1, 4>(buf, where, i0, i1, lane, staged, zero, part, blocks, a.stride, a.off);
        lds_barrier();
        // (units counted from the token's first)
        sums.add(split, j, max(u0, my0) - my0, min(u0 + nu, my1) - my0, [&](int u) {
            const int at = my0 + u;
            return weight_of[at / a.groups] * part[((at - u0) * nt + o_tile) * 16 + o_r];
        });
        lds_barrier();
    }
    const float sum = sums.total(split, outputs, red);
    if (tid < outputs) {
        const int64_t at = int64_t(o_m) * a.rows + 16 * (tile0 + o_tile) + o_r;
        a.out[at] = a.residual ? a.residual[at] + sum : sum;
    }
}

// Y[m] = residual[m] + the sum of the token's weighted rows, in choice order (pairs whose expert
// is out of range wrote none).
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ rows_of,
                                                          const int32_t* __restrict__ ids,
                                                          const float* residual, float* Y, int topk, int experts,
                                                          int K) {
    const int m = blockIdx.y;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (4 * c >= K) return;
    float4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < topk; ++j) {
        const int64_t p = int64_t(m) * topk + j;
        if (unsigned(ids[p]) >= unsigned(experts)) continue;
        const float4 v = reinterpret_cast<const float4*>(rows_of + p * K)[c];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    const int64_t at = int64_t(m) * K + 4 * c;
    if (residual) {
        const float4 r = *reinterpret_cast<const float4*>(residual + at);
        s.x += r.x; s.y += r.y; s.z += r.z; s.w += r.w;
    }
    *reinterpret_cast<float4*>(Y + at) = s;
}

// ------------------------------------------------------------------ launch
// f(integral_constant<int, type>)
template <class F>
hipError_t with_type(int type, F&& f) {
    switch (type) {
        case kQ4_0: return f(std::integral_constant<int, kQ4_0>{});
        case kQ4_1: return f(std::integral_constant<int, kQ4_1>{});
        case kQ5_0: return f(std::integral_constant<int, kQ5_0>{});
        case kQ5_1: return f(std::integral_constant<int, kQ5_1>{});
        case kQ8_0: return f(std::integral_constant<int, kQ8_0>{});
        case kQ4_K: return f(std::integral_constant<int, kQ4_K>{});
        case kQ5_K: return f(std::integral_constant<int, kQ5_K>{});
        case kQ6_K: return f(std::integral_constant<int, kQ6_K>{});
        default: return hipErrorInvalidValue;
    }
}

int64_t row_bytes_of(int type, BlockLayout lay, int64_t in) { return in / block_values_of(type) * lay.stride; }

template <bool UP>
hipError_t launch_group(int type, BlockLayout lay, MoeArgs a, bool pairs_mode, int cus, hipStream_t s) {
    constexpr int kMats = UP ? 2 : 1;
    a.stride = lay.stride;
    a.off = lay.off;
    a.row_bytes = row_bytes_of(type, lay, a.in);
    a.groups = (a.in + 255) / 256;
    const int slots = pairs_mode ? a.pairs : std::min(a.pairs, a.experts);
    const int tiles = a.rows / 16;
    // up to four tiles per workgroup while two workgroups per CU remain
    a.tiles = int(std::min<int64_t>(4, std::max<int64_t>(1, int64_t(slots) * tiles / (2 * cus))));
    const int T = pairs_mode ? 1 : kTokens;
    const int per_group = T * (kUnitBytes + a.tiles * kMats * 64);
    a.phase = std::max(1, std::min(a.groups, kStageBudget / per_group));
    const int list_room = pairs_mode ? 4 : (a.pairs + 3) & ~3;
    const size_t lds = 128 + kMoeMaxExperts / 8 + 16 + kThreads * 4 + size_t(list_room) * 4 + size_t(a.phase) * per_group;
    const dim3 grid((tiles + a.tiles - 1) / a.tiles, slots);
    return with_type(type, [&](auto qt) {
        constexpr int QT = decltype(qt)::value;
        if constexpr (UP) {
            if (pairs_mode) {
                hipLaunchKernelGGL((moe_group_kernel<QT, true, true>), grid, dim3(kThreads), lds, s, a);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((moe_group_kernel<QT, UP, false>), grid, dim3(kThreads), lds, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_down_pairs(int type, BlockLayout lay, MoeArgs a, hipStream_t s) {
    a.stride = lay.stride;
    a.off = lay.off;
    a.row_bytes = row_bytes_of(type, lay, a.in);
    a.groups = (a.in + 255) / 256;
    a.tiles = 1;
    const int per_unit = kUnitBytes + a.tiles * 64;
    a.phase = std::max(1, std::min(a.pairs * a.groups, kStageBudget / per_unit));
    const size_t lds = 128 + 16 + kThreads * 4 + kMoeFewPairs * 16 + 16 + size_t(a.phase) * per_unit;
    const dim3 grid((a.rows / 16 + a.tiles - 1) / a.tiles);
    return with_type(type, [&](auto qt) {
        constexpr int QT = decltype(qt)::value;
        hipLaunchKernelGGL((moe_down_pairs_kernel<QT>), grid, dim3(kThreads), lds, s, a);
        return hipGetLastError();
    });
}

#define MQ_MOE_INSTANCES(QT)                                          \
    template __global__ void moe_group_kernel<QT, true, true>(MoeArgs);   \
    template __global__ void moe_group_kernel<QT, true, false>(MoeArgs);  \
    template __global__ void moe_group_kernel<QT, false, false>(MoeArgs); \
    template __global__ void moe_down_pairs_kernel<QT>(MoeArgs);
MQ_MOE_INSTANCES(kQ4_0)
MQ_MOE_INSTANCES(kQ4_1)
MQ_MOE_INSTANCES(kQ5_0)
MQ_MOE_INSTANCES(kQ5_1)
MQ_MOE_INSTANCES(kQ8_0)
MQ_MOE_INSTANCES(kQ4_K)
MQ_MOE_INSTANCES(kQ5_K)
MQ_MOE_INSTANCES(kQ6_K)
#undef MQ_MOE_INSTANCES

size_t h_bytes(int64_t pairs, int64_t F) { return round_up256(size_t(pairs) * size_t(F) * 4); }

}  // namespace

// Few pairs (kMoeFewPairs): every pair is a slot of its own, and an expert that two tokens share
// is read twice (the second time from cache).
bool moe_few_pairs(int64_t pairs) { return pairs <= kMoeFewPairs; }

size_t moe_scratch_bytes(int64_t pairs, int64_t F, int64_t K) {
    return h_bytes(pairs, F) + (moe_few_pairs(pairs) ? 0 : round_up256(size_t(pairs) * size_t(K) * 4));
}

hipError_t moe_set_attributes(size_t lds_limit) {
    const int room = int(std::min(lds_limit, kGfx950LdsBytes));
    hipError_t e = hipSuccess;
    for (int type : {kQ4_0, kQ4_1, kQ5_0, kQ5_1, kQ8_0, kQ4_K, kQ5_K, kQ6_K})
        e = e != hipSuccess ? e : with_type(type, [&](auto qt) {
            constexpr int QT = decltype(qt)::value;
            const void* const kernels[] = {reinterpret_cast<const void*>(&moe_group_kernel<QT, true, true>),
                                           reinterpret_cast<const void*>(&moe_group_kernel<QT, true, false>),
                                           reinterpret_cast<const void*>(&moe_group_kernel<QT, false, false>),
                                           reinterpret_cast<const void*>(&moe_down_pairs_kernel<QT>)};
            hipError_t r = hipSuccess;
            for (const void* k : kernels)
                if (r == hipSuccess) r = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, room);
            return r;
        });
    return e;
}

hipError_t launch_moe_ffn(const MoeLayer& l, hipStream_t s, const char** name) {
    const int64_t pairs = l.M * l.topk;
    const bool few = moe_few_pairs(pairs);
    float* h = static_cast<float*>(l.scratch);
    float* rows = reinterpret_cast<float*>(static_cast<uint8_t*>(l.scratch) + h_bytes(pairs, l.F));
    *name = few ? "moe_pairs" : "moe_grouped";
    MoeArgs a = {};
    a.ids = l.ids;
    a.wts = l.wts;
    a.pairs = int(pairs);
    a.topk = int(l.topk);
    a.experts = int(l.E);
    a.act = l.act;
    a.w0 = l.Wg;
    a.w1 = l.Wu;
    a.x = l.X;
    a.out = h;
    a.in = int(l.K);
    a.rows = int(l.F);
    hipError_t e = launch_group<true>(l.gu_type, l.gu_layout, a, few, l.cu_count, s);
    if (e != hipSuccess) return e;
    a.w0 = l.Wd;
    a.w1 = nullptr;
    a.x = h;
    a.in = int(l.F);
    a.rows = int(l.K);
    if (few) {
        a.residual = l.residual;
        a.out = l.Y;
        return launch_down_pairs(l.d_type, l.d_layout, a, s);
    }
    a.out = rows;
    e = launch_group<false>(l.d_type, l.d_layout, a, false, l.cu_count, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned(l.K) / 4 + 255) / 256, unsigned(l.M)), dim3(256), 0, s, rows,
                       l.ids, l.residual, l.Y, int(l.topk), int(l.E), int(l.K));
    return hipGetLastError();
}

}  // namespace mq
