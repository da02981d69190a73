// mq_moe_ffn: a mixture-of-experts feed-forward layer for a few tokens,
//   Y[m] = residual[m] + sum_j w[m][j] * Wd_e ( act(Wg_e X[m]) * (Wu_e X[m]) ),   e = ids[m][j],
// over block-quantized expert weights and f32 activations.  (token, choice) pairs p = m k + j.
//
// What bounds it.  A few tokens touch each weight of a chosen expert only once or a few
// times, so the floor is the chosen experts' bytes from HBM; everything here is arranged to
// keep weight loads in flight and to spend few instructions per weight.
//
// Split.  Two launches at least, because every output of the down product needs every h of its token.
//   One token: `up`, a workgroup per (choice, a few 16-row tiles of F) that forms act(g) * u where both sums
//   meet, h f32 [choice][F] to scratch; `down`, a workgroup per 16 rows of Y for every choice, which
//   adds the choices itself (nothing is exchanged between workgroups).
//   More tokens: a slot is up to `set` tokens of one chosen expert, whose weights are read once for all
//   of them; `up` leaves the gate and the up sums, `down` the weighted rows of every pair, and a
//   third launch adds a token's rows in choice order.  (Two tokens already gain from it: 64 experts of
//   2048 x 1024, 8 choices, Q4_K: 21.9 us, four tokens 32.3, eight 48.8, where the one-token kernels
//   extended to few tokens took 37.8, 65.5 and 109.  The third launch's work in the down kernel's last
//   workgroups instead was slower: eight tokens 51.3 -> 62.2.)
//
// Arithmetic.  The exact-integer scheme of the GEMV kernels: per 32-value block of the
// activations x = 2^-s v with v an integer of at most 22 bits (relative to the block's largest
// value the staged x is off by at most 2^-22), v = 65536 d2 + 256 d1 + d0 in signed bytes.
// One v_mfma_i32_16x16x32_i8 per 32-value block multiplies four tokens:
//   A (16 x 32): row 4 t + p (p < 3) = digit plane p of token t (row 4 t + 3 repeats plane 2),
//   B (32 x 16): column n = the block's 32 codes of weight row n; lane (n, q) holds eight of them,
// so lane (n, q) receives the three plane sums of token q and row n (all exact), combines them and
// applies the block's scale in f32.  A wave walks the 256-value groups of its 16 rows with one f32
// accumulator per four tokens; nothing crosses lanes.  (Q6_K's scales change every 16 values: a
// second product over A's first 16 values gives the first half, the difference the second.)
// The same work for one token wastes three quarters of the matrix rows, which have the room: one
// token's vector work is about 100 instructions per 2304 weight bytes, 40% of the time those bytes take
// from HBM.
//
// Weights: a wave reads one group of its 16 rows at a time as whole 16-byte chunks, consecutive lanes on
// consecutive chunks, into registers, kDepth groups ahead, and passes each through LDS of its own,
// where every lane picks the bytes its operands need.  (Loading those 8-byte pieces straight from
// memory, 16 rows apart, kept the address path busy for most of the time the bytes take from HBM:
// 48 tokens, 4096 x 1536 Q4_K gate and up, 348 us.)
#include <algorithm>
#include <type_traits>

#include "mq_device.h"
#include "mq_epilogue.h"
#include "mq_internal.h"
#include "weight_units.h"

namespace mq {

// The kernels of one token: at most kMoeOneTopk choices.
static bool moe_one(int64_t M, int64_t topk) { return M == 1 && topk <= kMoeOneTopk; }

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kFracBits = 22;
constexpr int kPlane = 272;                  // bytes of a staged digit plane: 256 and 16, so that the twelve planes of
                                             // four tokens start in different quads of the 64 LDS banks
constexpr int kPlanes = 3 * kPlane;
constexpr int kDepth = 2;                    // weight groups in flight per wave (48 tokens: 421 us; with 4, 448)
constexpr int kOneUpWaves = 4096;            // waves of the one-token up kernel
constexpr int kManyFixed = 48 + 16 * kWaves;  // many tokens: LDS of the slot's lists

// A wave-uniform pointer to device memory held in scalar registers: a load from it plus a 32-bit lane
// offset then takes one vector register for its address (the compiler otherwise keeps a 64-bit pointer
// per lane for every load of the loop, and runs out of registers).  It stays a global pointer: a flat
// load would be waited for with every LDS read.
typedef const __attribute__((address_space(1))) uint8_t* global_bytes;
__device__ __forceinline__ global_bytes scalar(const uint8_t* p) {
    global_bytes g = (global_bytes)p;
    asm("" : "+s"(g));
    return g;
}

// LDS writes of every wave visible, without waiting for global loads in flight
// (__syncthreads waits for those too).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// ------------------------------------------------------------------ weights
// A code is unsigned with an offset, taken off through the integer sum of v
template <int QT> constexpr int code_offset() { return QT == kQ6_K ? 32 : QT == kQ4_0 ? 8 : QT == kQ5_0 ? 16 : 0; }
// Whether |sum code v| over a block can pass 2^31 (the plane sums are then combined in f32): 5-bit codes
// without an offset and 8-bit codes.  (The others: 32 * 15 * 2^22 < 2^31; with the offset taken
// off, modulo 2^32, 16 * 32 * (2^22 - 1) and 32 * 16 * (2^22 - 1) < 2^31.)
template <int QT> constexpr bool wide_sums() { return QT == kQ8_0 || QT == kQ5_K || QT == kQ5_1; }

// Lane (n, q)'s part of one 256-value group of weight row n: of each of the eight 32-value blocks
// eight codes as MFMA B bytes, which the blocks' layouts order differently:
//   K-quants and Q8_0: values 8 q .. 8 q + 7 of the block;
//   Q4_0, Q4_1, Q5_0, Q5_1: values 4 q .. 4 q + 3 and 16 + 4 q .. 16 + 4 q + 3 (a nibble pair per byte)
// (the staged activations are in the same order), and each block's scale and minimum:
//   weight = d * sc[b] * code - dm * mn[b]   (Q6_K: sc[2 b + half of the block]).
template <int QT>
struct Group {
    static constexpr int kScales = QT == kQ6_K ? 16 : 8;
    uint64_t codes[8];
    float sc[kScales];
    float mn[8];
    float d, dm;
};

// Bytes of a group of a row, and the 16-byte chunks that cover it from any even start (K-quants of
// 16-byte blocks: from a 16-byte boundary), in the GGUF payload or in the slots mq_repack writes.
template <int QT> constexpr bool whole_chunks() { return QT == kQ4_K || QT == kQ5_K; }
template <int QT> constexpr int group_bytes() { return 8 * Legacy<QT>::kBytes; }
template <> constexpr int group_bytes<kQ4_K>() { return 144; }
template <> constexpr int group_bytes<kQ5_K>() { return 176; }
template <> constexpr int group_bytes<kQ6_K>() { return 224; }   // 210 from any even start, or a 224-byte slot
template <> constexpr int group_bytes<kQ8_0>() { return 288; }   // 272 bytes, or eight 36-byte slots
template <int QT>
constexpr int row_chunks() {
    constexpr bool covered = whole_chunks<QT>() || QT == kQ6_K;
    return (group_bytes<QT>() + (covered ? 0 : 14) + 15) / 16;
}

// One group of a wave's 16 rows: chunk c (row c / row_chunks, 16 bytes c % row_chunks of the row's
// group) in register c / 64 of lane c % 64, then in its row of the wave's LDS slot.
template <int QT>
struct Tile {
    static constexpr int kRow = (row_chunks<QT>() | 1) * 16;   // LDS bytes of a row: an odd number of bank quads, so
                                                               // that the 16 rows' start in different ones
    static constexpr bool kPadded = kRow != row_chunks<QT>() * 16;
    static constexpr int kSlot = 16 * kRow;
    static constexpr int kChunks = 16 * row_chunks<QT>();
    static constexpr int kLoads = (kChunks + 63) / 64;
    v4u r[kLoads];

    // lane constants: byte offsets of its chunks' rows in the tile, and of the chunks in the row
    struct Lane {
        uint32_t row[kLoads], col[kLoads], at[kLoads];   // (at: its byte in the slot)
        __device__ Lane(int lane, uint32_t row_bytes) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int c = min(lane + 64 * i, kChunks - 1);
                row[i] = uint32_t(c / row_chunks<QT>()) * row_bytes;
                col[i] = uint32_t(c % row_chunks<QT>()) * 16;
                at[i] = kPadded ? uint32_t(c / row_chunks<QT>()) * kRow + col[i] : uint32_t(lane + 64 * i) * 16;
            }
        }
    };
    // `tile`: the tile's first byte (16-byte aligned, 16 row_bytes long); `at`: the group's byte in a row.
    // Chunks past the tile (they hold none of the rows' bytes) read its last one.
    __device__ void load(const uint8_t* tile, const Lane& l, uint32_t at, uint32_t tile_bytes) {
        const global_bytes b = scalar(tile);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint32_t o = l.row[i] + at;
            if constexpr (!whole_chunks<QT>()) o = min(o & ~15u, tile_bytes - 16 - l.col[i]);
            r[i] = *(const __attribute__((address_space(1))) v4u*)(b + (o + l.col[i]));
        }
    }
    __device__ void store(uint8_t* slot, int lane, const Lane& l) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (64 * (i + 1) <= kChunks || lane + 64 * i < kChunks)
                *reinterpret_cast<v4u*>(slot + l.at[i]) = r[i];
    }
};

// LDS reads of 4 and 8 bytes at even byte `at` of a row (which starts on a dword), as the dwords that
// hold them.
__device__ __forceinline__ uint32_t even4(const uint8_t* row, uint32_t at) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + (at >> 2);
    return align_byte(w[1], w[0], at & 3u);
}
__device__ __forceinline__ uint64_t even8(const uint8_t* row, uint32_t at) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(row) + (at >> 2);
    return (uint64_t(align_byte(w[2], w[1], at & 3u)) << 32) | align_byte(w[1], w[0], at & 3u);
}
__device__ __forceinline__ uint32_t even2(const uint8_t* row, uint32_t at) {
    return *reinterpret_cast<const uint16_t*>(row + at);
}

// decode(o, b, s, q, g, blocks, stride): lane (n, q)'s operands of a group whose bytes start at byte s
// (even, below 16) of its row's chunks b in LDS.

// The eight 6-bit (scale, min) pairs of a Q4_K / Q5_K header, and d, dmin.
template <class G>
__device__ __forceinline__ void header(G& o, const uint4 hd) {
    const uint32_t sc0 = hd.y & 0x3F3F3F3Fu, mn0 = hd.z & 0x3F3F3F3Fu;
    const uint32_t sc1 = (hd.w & 0x0F0F0F0Fu) | ((hd.y >> 2) & 0x30303030u);
    const uint32_t mn1 = ((hd.w >> 4) & 0x0F0F0F0Fu) | ((hd.z >> 2) & 0x30303030u);
    o.sc[0] = ubyte_f<0>(sc0); o.sc[1] = ubyte_f<1>(sc0); o.sc[2] = ubyte_f<2>(sc0); o.sc[3] = ubyte_f<3>(sc0);
    o.sc[4] = ubyte_f<0>(sc1); o.sc[5] = ubyte_f<1>(sc1); o.sc[6] = ubyte_f<2>(sc1); o.sc[7] = ubyte_f<3>(sc1);
    o.mn[0] = ubyte_f<0>(mn0); o.mn[1] = ubyte_f<1>(mn0); o.mn[2] = ubyte_f<2>(mn0); o.mn[3] = ubyte_f<3>(mn0);
    o.mn[4] = ubyte_f<0>(mn1); o.mn[5] = ubyte_f<1>(mn1); o.mn[6] = ubyte_f<2>(mn1); o.mn[7] = ubyte_f<3>(mn1);
    o.d = half_bits_to_float(hd.x & 0xFFFFu);
    o.dm = half_bits_to_float(hd.x >> 16);
}

__device__ __forceinline__ void decode(Group<kQ4_K>& o, const uint8_t* b, uint32_t s, int q, int, int, int) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t c = *reinterpret_cast<const uint64_t*>(b + 16 + 32 * i + 8 * q);
        o.codes[2 * i] = c & 0x0F0F0F0F0F0F0F0Full;
        o.codes[2 * i + 1] = (c >> 4) & 0x0F0F0F0F0F0F0F0Full;
    }
    header(o, *reinterpret_cast<const uint4*>(b));
}

__device__ __forceinline__ void decode(Group<kQ5_K>& o, const uint8_t* b, uint32_t s, int q, int, int, int) {
    const uint64_t h = *reinterpret_cast<const uint64_t*>(b + 16 + 8 * q);   // bit i of byte l: bit 4 of value l of block i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t c = *reinterpret_cast<const uint64_t*>(b + 48 + 32 * (i / 2) + 8 * q);
        const uint64_t low = (i & 1) ? c >> 4 : c;
        const uint64_t high = i < 4 ? h << (4 - i) : h >> (i - 4);
        o.codes[i] = (low & 0x0F0F0F0F0F0F0F0Full) | (high & 0x1010101010101010ull);
    }
    header(o, *reinterpret_cast<const uint4*>(b));
}

// Block 4 h + r of Q6_K: half h, run r; low bits in ql[64 h + 32 (r % 2) ..], nibble r / 2, high bits
// at bit 2 r of qh[32 h ..]; the sub-scales of its two 16-value halves are scales[8 h + 2 r ..].
__device__ __forceinline__ void decode(Group<kQ6_K>& o, const uint8_t* b, uint32_t s, int q, int, int, int) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t qh = even8(b, s + 128 + 32 * h + 8 * q);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t ql = even8(b, s + 64 * h + 32 * k + 8 * q);
            // runs k (low nibbles) and k + 2 (high nibbles)
            const uint64_t h0 = k == 0 ? qh << 4 : qh << 2, h1 = k == 0 ? qh : qh >> 2;
            o.codes[4 * h + k] = (ql & 0x0F0F0F0F0F0F0F0Full) | (h0 & 0x3030303030303030ull);
            o.codes[4 * h + k + 2] = ((ql >> 4) & 0x0F0F0F0F0F0F0F0Full) | (h1 & 0x3030303030303030ull);
        }
        const uint64_t sub = even8(b, s + 192 + 8 * h);
        const uint32_t sw[2] = {uint32_t(sub), uint32_t(sub >> 32)};
#pragma unroll
        for (int i = 0; i < 8; ++i) o.sc[8 * h + i] = float(int32_t(sw[i >> 2] << (24 - 8 * (i & 3))) >> 24);
    }
    o.d = half_bits_to_float(even2(b, s + 208));
    o.dm = 0.f;
}

// The 32-value types: block 8 g + i of the row.  In a last group of fewer than eight blocks those past
// the row's end are its last block again (their staged activations are zero).
__device__ __forceinline__ void decode(Group<kQ8_0>& o, const uint8_t* b, uint32_t s, int q, int g, int blocks,
                                       int stride) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = s + stride * min(i, blocks - 1 - 8 * g);
        o.codes[i] = even8(b, p + 2 + 8 * q);
        o.sc[i] = half_bits_to_float(even2(b, p));
    }
    o.d = 1.f;
    o.dm = 0.f;
}

template <int QT>
__device__ __forceinline__ void decode(Group<QT>& o, const uint8_t* b, uint32_t s, int q, int g, int blocks, int) {
    using L = Legacy<QT>;
    constexpr int at = L::kMin ? 4 : 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = s + L::kBytes * min(i, blocks - 1 - 8 * g);
        const uint32_t c = even4(b, p + at + (L::kHigh ? 4 : 0) + 4 * q);
        uint32_t lo = c & 0x0F0F0F0Fu, hi = (c >> 4) & 0x0F0F0F0Fu;
        if constexpr (L::kHigh) {
            const uint32_t h = even4(b, p + at) >> (4 * q);   // bits 0..3 and 16..19: this lane's values
            lo |= spread4(h & 15u) << 4;
            hi |= spread4((h >> 16) & 15u) << 4;
        }
        o.codes[i] = (uint64_t(hi) << 32) | lo;
        o.sc[i] = half_bits_to_float(even2(b, p));
        o.mn[i] = L::kMin ? half_bits_to_float(even2(b, p + 2)) : 0.f;
    }
    o.d = 1.f;
    o.dm = -1.f;
}

// ------------------------------------------------------------------ staged activations
// `count` tokens' 256 values of one group in LDS, count * unit_bytes: the digit planes of every token
// (kPlanes each, plane p at kPlane p), then the f32 scales 2^-s of every token's eight blocks (32
// bytes each), then what the type needs of the integer sums of v (32 or, Q6_K, 64 bytes each):
//   types with a minimum: f32 2^-s sum(v) per block; Q4_0, Q5_0: int32 offset * sum(v) per block;
//   Q6_K: int32 32 sum(v) per 16-value half, half i of block b at 2 b + i.
// All of them come from the same rounded v that the digits hold, so a code's offset or a
// minimum multiplies exactly the x that the codes meet.  A block that holds an infinity or a
// NaN has a NaN scale: every output of that token becomes NaN.
template <int QT> constexpr int sum_bytes() { return QT == kQ6_K ? 64 : 32; }
template <int QT> constexpr int unit_bytes() { return kPlanes + 32 + sum_bytes<QT>(); }

__device__ __forceinline__ uint32_t digits3(int v) { return (uint32_t(v) + 0x00808080u) ^ 0x00808080u; }

// Stage token t's 256 values: lane l holds values 4l .. 4l + 3 (zeros past the row's end).
template <int QT>
__device__ __forceinline__ void stage_token(uint8_t* group, int t, int count, const float4 x, int lane) {
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
    // the lane's dword of its block, in the order of the B bytes
    const int b = lane >> 3, k = lane & 7;
    const int pos = 8 * b + (Legacy<QT>::kIs ? (k < 4 ? 2 * k : 2 * k - 7) : k);
    uint32_t* planes = reinterpret_cast<uint32_t*>(group + t * kPlanes) + pos;
    planes[0] = __builtin_amdgcn_perm(t23, t01, 0x05040100u);
    planes[kPlane / 4] = __builtin_amdgcn_perm(t23, t01, 0x07060302u);
    planes[kPlane / 2] = __builtin_amdgcn_perm(u23, u01, 0x05040100u);
    float* scl = reinterpret_cast<float*>(group + count * kPlanes + t * 32);
    // (0 * x is NaN for an infinity or a NaN and 0 otherwise; a sum keeps the NaN)
    float bad = 0.f * x.x + 0.f * x.y + (0.f * x.z + 0.f * x.w);
    bad = lanes8_sum(bad);
    const float scale = ldexpf(1.0f, -s) + bad;
    if (k == 0) scl[b] = scale;
    uint8_t* sums = group + count * (kPlanes + 32) + t * sum_bytes<QT>();
    int sum = (v0 + v1) + (v2 + v3);
    if constexpr (QT == kQ6_K) {
        sum = lanes8_sum<2>(sum);
        if ((k & 3) == 0) reinterpret_cast<int*>(sums)[2 * b + (k >> 2)] = code_offset<QT>() * sum;
    } else if constexpr (code_offset<QT>() != 0) {
        sum = lanes8_sum(sum);
        if (k == 0) reinterpret_cast<int*>(sums)[b] = code_offset<QT>() * sum;
    } else if constexpr (has_min_term<QT>()) {
        sum = lanes8_sum(sum);
        if (k == 0) reinterpret_cast<float*>(sums)[b] = float(sum) * scale;
    }
}

// ------------------------------------------------------------------ products
// What a lane reads of a staged group of `count` tokens for tokens 4 S .. 4 S + 3: its A row's digits of
// each block, and the scales and sums of token 4 S + q.  (Tokens past the last are the last again;
// their results are not used.)
template <int QT>
struct LaneTokens {
    int a;       // byte offset of the A row's digits of block 0 (+ 32 b)
    int scale;   // of the token's block scales
    int sums;
    __device__ LaneTokens(int lane, int set, int count) {
        const int row = lane & 15, q = lane >> 4;
        const int ta = min(4 * set + (row >> 2), count - 1), tq = min(4 * set + q, count - 1);
        a = ta * kPlanes + min(row & 3, 2) * kPlane + 8 * q;
        scale = count * kPlanes + tq * 32;
        sums = count * (kPlanes + 32) + tq * sum_bytes<QT>();
    }
};

// acc += the group's share of the dot product of weight row n with token 4 S + q
template <int QT>
__device__ __forceinline__ float group_dot(const Group<QT>& w, const uint8_t* staged, const LaneTokens<QT>& l, float acc) {
    const v4i z = {0, 0, 0, 0};
    float s[8];
    *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(staged + l.scale);
    *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(staged + l.scale + 16);
    constexpr int kSums = QT == kQ6_K ? 16 : 8;
    union {
        int i[kSums];
        float f[kSums];
    } sum;
    if constexpr (code_offset<QT>() != 0 || has_min_term<QT>()) {
#pragma unroll
        for (int i = 0; i < kSums; i += 4)
            *reinterpret_cast<int4*>(sum.i + i) = *reinterpret_cast<const int4*>(staged + l.sums + 4 * i);
    }
    // the three plane sums as one integer, modulo 2^32
    auto joined = [](const v4i& c) { return (((uint32_t(c[2]) << 8) + uint32_t(c[1])) << 8) + uint32_t(c[0]); };
    float codes = 0.f, mins = 0.f;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const long a = *reinterpret_cast<const long*>(staged + l.a + 32 * b);
        const v4i c = __builtin_amdgcn_mfma_i32_16x16x32_i8(a, long(w.codes[b]), z, 0, 0, 0);
        if constexpr (QT == kQ6_K) {
            // lane groups 0 and 1 hold the block's first 16 values
            const long first = (threadIdx.x & 32) ? 0l : a;
            const v4i c1 = __builtin_amdgcn_mfma_i32_16x16x32_i8(first, long(w.codes[b]), z, 0, 0, 0);
            const uint32_t all = joined(c), one = joined(c1);
            const float f1 = float(int(one - uint32_t(sum.i[2 * b])));
            const float f2 = float(int(all - one - uint32_t(sum.i[2 * b + 1])));
            codes = fmaf(fmaf(w.sc[2 * b], f1, w.sc[2 * b + 1] * f2), s[b], codes);
        } else {
            float f;
            if constexpr (wide_sums<QT>()) {
                f = fmaf(float((c[2] << 8) + c[1]), 256.0f, float(c[0]));   // (|256 c2 + c1| < 2^28)
            } else if constexpr (code_offset<QT>() != 0) {
                f = float(int(joined(c) - uint32_t(sum.i[b])));
            } else {
                f = float(int(joined(c)));
            }
            codes = fmaf(f * s[b], w.sc[b], codes);
            if constexpr (has_min_term<QT>()) mins = fmaf(sum.f[b], w.mn[b], mins);
        }
    }
    if constexpr (has_min_term<QT>()) acc = fmaf(-w.dm, mins, acc);
    return fmaf(w.d, codes, acc);
}

struct MoeArgs {
    const uint8_t* w0;     // up: gate weights; down: down weights
    const uint8_t* w1;     // up: up weights
    const float* x;        // up: X [M][in]; down: h [choice][in], or its factors, each [pair][in]
    const int32_t* ids;    // [pairs]
    const float* wts;      // [pairs] (down)
    const float* residual; // [rows] or null (down, one token)
    float* out;            // one token: h [choice][rows], Y [rows]; else the factors [pair][rows] each, weighted rows
    int pairs, topk, experts;
    int in, rows;          // values per weight row, weight rows per expert
    int groups;            // 256-value groups per row
    int splits;            // one token: waves that share a tile's groups (part ks: groups ks, ks + splits, ..)
    int set;               // many tokens: tokens staged together
    int act;
    int stride, off;       // weight block layout
    int64_t row_bytes;
};

template <int QT>
__device__ __forceinline__ int row_blocks(int in) {
    return QT == kQ4_K || QT == kQ5_K || QT == kQ6_K ? in >> 8 : in >> 5;
}

// Block slots of a 256-value group.
template <int QT>
constexpr int row_blocks_per_group() {
    return QT == kQ4_K || QT == kQ5_K || QT == kQ6_K ? 1 : 8;
}

// ------------------------------------------------------------------ many tokens
// blockIdx.y: a slot, `set` (at most four) tokens of one chosen expert; the expert's units (16 rows of
// one matrix) are dealt to the waves of the gridDim.x workgroups.  A workgroup stages all groups of the
// slot's tokens, then every wave walks its units by itself: nothing but the staging needs a barrier,
// and the stream of weights does not stop between units.  The slots of an expert of more
// tokens read the same weights at about the same time (from HBM once).
// (48 tokens, 8 of 128 experts each, 4096 x 1536, graph replay: up Q4_K 212 us, 4.1 TB/s of chosen
// weights; down Q6_K 186 us, 3.4 TB/s.  By the counters the vector ALU issues 60% (Q6_K 75%) of the time:
// decoding a group and joining its plane sums.  LDS bank conflicts are 11% and 15%, 20% and 35% before
// planes and rows were padded to odd bank quads, 429 -> 414 us for the layer.)
//   up    leaves the gate and the up sums, f32 [pair][F] each: act(g) * u is formed where the down
//         kernel stages h, so that a wave's unit is one matrix's 16 rows (at 48 tokens, 4096 x 1536,
//         the last round of waves is then 1 of 7 and not 1 of 4)
//   down  leaves the weighted rows, f32 [pair][K].

// A slot's pairs (as slot_pairs_of below) for at most 64 pairs, a lane each, in every wave by itself (no trip through LDS, no barrier):
// slots in the order of their first pairs; `list` is the wave's own.
__device__ __forceinline__ int slot_pairs_of_64(const MoeArgs& a, int lane, int* count, int* list) {
    const int e = lane < a.pairs ? a.ids[lane] : -1;
    const bool valid = unsigned(e) < unsigned(a.experts);
    unsigned long long same = __ballot(valid);   // the lanes of this lane's expert
#pragma unroll
    for (int b = 1; b < kMoeMaxExperts; b <<= 1) {
        const unsigned long long m = __ballot((e & b) != 0);
        same &= (e & b) ? m : ~m;
    }
    const unsigned long long below = (1ull << lane) - 1;
    const int rank = __popcll(same & below);
    const unsigned long long heads = __ballot(valid && rank % a.set == 0);   // a slot's first pair each
    const bool mine = valid && rank % a.set == 0 && __popcll(heads & below) == int(blockIdx.y);
    const unsigned long long head = __ballot(mine);
    if (head == 0) return -1;
    const int src = __builtin_amdgcn_readfirstlane(__ffsll(head) - 1);
    const int expert = __builtin_amdgcn_readlane(e, src), first = __builtin_amdgcn_readlane(rank, src);
    const bool in = valid && e == expert && rank >= first && rank < first + a.set;
    if (in) list[rank - first] = lane;
    *count = __popcll(__ballot(in));
    return expert;
}

// Slot blockIdx.y: its expert (-1: there are fewer slots), and its pairs in list[0 .. *count - 1].
// LDS: counts [kMoeMaxExperts], tmp [16], list.  Slots are numbered expert by expert.
__device__ __forceinline__ int slot_pairs_of(const MoeArgs& a, int* counts, int* tmp, int* count, int* list) {
    static_assert(kMoeMaxExperts <= kThreads, "a thread per expert");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    counts[tid] = 0;
    if (tid == 0) tmp[8] = -1;
    lds_barrier();
    for (int p = tid; p < a.pairs; p += kThreads) {
        const int e = a.ids[p];
        if (unsigned(e) < unsigned(a.experts)) atomicAdd(&counts[e], 1);
    }
    lds_barrier();
    // slots before expert tid's: a scan over the wave, then over the waves
    const int mine = (counts[tid] + a.set - 1) / a.set;
    int before = mine;
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(before, off, 64);
        if (lane >= off) before += v;
    }
    if (lane == 63) tmp[wave] = before;
    lds_barrier();
    for (int w = 0; w < wave; ++w) before += tmp[w];
    before -= mine;
    const int s = int(blockIdx.y) - before;
    if (s >= 0 && s < mine) {
        tmp[8] = tid;
        tmp[9] = s * a.set;                                   // rank of the slot's first pair
        *count = min(a.set, counts[tid] - s * a.set);
    }
    lds_barrier();
    const int expert = __builtin_amdgcn_readfirstlane(tmp[8]);
    if (expert < 0) return expert;
    // ranks of the expert's pairs: wave w takes a consecutive part of them
    const int first = tmp[9];
    const int per = ((a.pairs + kWaves - 1) / kWaves + 63) & ~63;
    const int p0 = wave * per, p1 = min(a.pairs, p0 + per);
    int n = 0;
    for (int p = p0 + lane; p - lane < p1; p += 64) n += __popcll(__ballot(p < p1 && a.ids[p] == expert));
    lds_barrier();
    if (lane == 0) tmp[wave] = n;
    lds_barrier();
    int rank = -first;
    for (int w = 0; w < wave; ++w) rank += tmp[w];
    for (int p = p0 + lane; p - lane < p1; p += 64) {
        const bool is = p < p1 && a.ids[p] == expert;
        const unsigned long long m = __ballot(is);
        const int r = rank + __popcll(m & ((1ull << lane) - 1));
        if (is && r >= 0 && r < a.set) list[r] = p;
        rank += __popcll(m);
    }
    lds_barrier();
    return expert;
}

template <int QT, bool UP>
__global__ __launch_bounds__(kThreads, 4) void moe_many_kernel(MoeArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* tmp = reinterpret_cast<int*>(smem);   // of slot_pairs_of, with the count; then a list of four per wave
    int* count_lds = tmp + 10;
    uint8_t* slots = smem + kManyFixed;
    uint8_t* staged = slots + kWaves * Tile<QT>::kSlot;
    int* counts = reinterpret_cast<int*>(slots);   // (before the first weights)
    static_assert(kWaves * Tile<QT>::kSlot >= kMoeMaxExperts * 4, "room for the counts");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q = lane >> 4;
    const bool few = a.pairs <= 64;
    int* list = tmp + 12 + (few ? 4 * wave : 0);
    int expert, count;
    if (few) {
        expert = slot_pairs_of_64(a, lane, &count, list);
        __builtin_amdgcn_wave_barrier();
    } else {
        expert = slot_pairs_of(a, counts, tmp, count_lds, list);
        count = __builtin_amdgcn_readfirstlane(*count_lds);
    }
    if (expert < 0) return;   // (uniform)

    constexpr int kMats = UP ? 2 : 1;
    const int units = (a.rows >> 4) * kMats, stride = int(gridDim.x) * kWaves;
    const int unit0 = int(blockIdx.x) * kWaves + wave;
    const int blocks = row_blocks<QT>(a.in);
    const uint32_t row_bytes = uint32_t(a.row_bytes), tile_bytes = 16 * row_bytes;
    const uint32_t group_step = uint32_t(row_blocks_per_group<QT>() * a.stride);
    const typename Tile<QT>::Lane lanes(lane, row_bytes);
    uint8_t* slot = slots + wave * Tile<QT>::kSlot;
    const int64_t expert_at = int64_t(expert) * a.rows * a.row_bytes;
    const int unit_size = count * unit_bytes<QT>();

    struct Cursor {
        int unit, g;
    };
    auto step = [&](Cursor& c) {
        if (++c.g == a.groups) {
            c.g = 0;
            c.unit += stride;
        }
    };
    Cursor ld = {min(unit0, units - 1), 0}, cp = {unit0, 0};
    Tile<QT> buf[kDepth];
    // (past the last unit: its last group again)
    auto load = [&](auto slot_c) __attribute__((always_inline)) {
        const uint8_t* w = (UP && (ld.unit & 1) ? a.w1 : a.w0) + expert_at + int64_t(UP ? ld.unit >> 1 : ld.unit) * tile_bytes;
        buf[decltype(slot_c)::value].load(w, lanes, uint32_t(ld.g) * group_step, tile_bytes);
        Cursor next = ld;
        step(next);
        if (next.unit < units) ld = next;
    };
    // Stage the tokens: (group, token), dealt to the waves in batches.  The first batch's activations are
    // requested before the first weights (a wave's loads return in order), and those before it is staged.
    const int staging = a.groups * count;
    constexpr int kBatch = UP ? 4 : 2;
    float4 x[kBatch], y[kBatch];
    auto fetch = [&](int u0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = min(u0 + kWaves * i, staging - 1);
            const int g = u / count, pair = list[u - g * count];
            const int k0 = 256 * g + 4 * lane;
            x[i] = y[i] = float4{0.f, 0.f, 0.f, 0.f};
            if (k0 < a.in) {
                const float* p = a.x + int64_t(UP ? pair / a.topk : pair) * a.in + k0;
                x[i] = *reinterpret_cast<const float4*>(p);
                if constexpr (!UP) y[i] = *reinterpret_cast<const float4*>(p + int64_t(a.pairs) * a.in);
            }
        }
    };
    auto stage = [&](int u0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + kWaves * i;
            const int g = u / count;
            if (u < staging) {
                float4 h = x[i];
                if constexpr (!UP) {
                    h.x = activate(h.x, a.act) * y[i].x;
                    h.y = activate(h.y, a.act) * y[i].y;
                    h.z = activate(h.z, a.act) * y[i].z;
                    h.w = activate(h.w, a.act) * y[i].w;
                }
                stage_token<QT>(staged + g * unit_size, u - g * count, count, h, lane);
            }
        }
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    static_assert(kDepth == 2, "the loops below name the slots");
    fetch(wave);
    load(S0{});
    load(S1{});
    stage(wave);
    for (int u0 = wave + kWaves * kBatch; u0 < staging; u0 += kWaves * kBatch) {
        fetch(u0);
        stage(u0);
    }
    const LaneTokens<QT> at(lane, 0, count);
    const int pair = list[min(q, count - 1)];
    const float weight = UP ? 1.f : a.wts[pair];
    float* out = a.out + int64_t(pair) * a.rows + n;
    float acc = 0.f;
    auto compute = [&](auto slot_c) __attribute__((always_inline)) {
        // (one wave's LDS operations complete in order: the reads see these writes, and the next
        // writes come after the reads)
        buf[decltype(slot_c)::value].store(slot, lane, lanes);
        __builtin_amdgcn_wave_barrier();
        const uint32_t start =
            whole_chunks<QT>() ? 0u : a.off + ((uint32_t(n) * row_bytes + uint32_t(cp.g) * group_step) & 15u);
        Group<QT> w;
        decode(w, slot + n * Tile<QT>::kRow, start, q, cp.g, blocks, a.stride);
        acc = group_dot<QT>(w, staged + cp.g * unit_size, at, acc);
        __builtin_amdgcn_wave_barrier();
        if (cp.g == a.groups - 1) {
            if (q < count) {
                if constexpr (UP) out[int64_t(cp.unit & 1) * a.pairs * a.rows + 16 * (cp.unit >> 1)] = acc;
                else out[16 * cp.unit] = weight * acc;
            }
            acc = 0.f;
        }
        step(cp);
    };
    lds_barrier();
    if (unit0 < units) {
        while (true) {
            compute(S0{});
            if (cp.unit >= units) break;
            load(S0{});
            compute(S1{});
            if (cp.unit >= units) break;
            load(S1{});
        }
    }
}

// ------------------------------------------------------------------ one token
// (8 of 64 experts of 2048 x 1024, Q4_K: up 7.4 us, down 6.7, 2.5 and 1.4 TB/s: two launches' ramps and
// round trips, and a down kernel of K / 16 = 128 workgroups, which leaves half of the 256 CUs idle.
// 4 of 32 of 4096 x 2048, 256 workgroups in down: up Q4_K 10.6 us, down Q6_K 9.6, 3.6 and 2.9 TB/s.)
// blockIdx.y: choice; blockIdx.x: kWaves / (2 splits) 16-row tiles of its expert.  Wave w: part w % splits of
// the groups (part ks: ks, ks + splits, ...) of matrix w / splits % 2 (gate, up), tile w / (2 splits) of
// the workgroup; the sums meet in LDS, parts in order.
template <int QT>
__global__ __launch_bounds__(kThreads, 4) void moe_one_up_kernel(MoeArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem);   // [wave][16 rows]
    uint8_t* slots = smem + kWaves * 64;
    uint8_t* staged = slots + kWaves * Tile<QT>::kSlot;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q = lane >> 4;
    // x is requested before anything that depends on the choice: group `wave` of it
    auto group_x = [&](int g) {
        const int k0 = 256 * g + 4 * lane;
        float4 v = {0.f, 0.f, 0.f, 0.f};
        if (k0 < a.in) v = *reinterpret_cast<const float4*>(a.x + k0);
        return v;
    };
    const float4 x0 = group_x(wave);
    const int expert = __builtin_amdgcn_readfirstlane(a.ids[blockIdx.y]);
    if (unsigned(expert) >= unsigned(a.experts)) return;   // (uniform) not this layer's: adds nothing
    const int tiles_wg = kWaves / (2 * a.splits);
    const int ks = wave % a.splits, mat = wave / a.splits & 1, wtile = wave / (2 * a.splits);
    const int tile = blockIdx.x * tiles_wg + wtile;
    const bool active = 16 * tile < a.rows;
    const int blocks = row_blocks<QT>(a.in);
    const uint8_t* const w =
        (mat ? a.w1 : a.w0) + (int64_t(expert) * a.rows + 16 * (active ? tile : 0)) * a.row_bytes;
    const uint32_t row_bytes = uint32_t(a.row_bytes), tile_bytes = 16 * row_bytes;
    const uint32_t group_step = uint32_t(row_blocks_per_group<QT>() * a.stride);
    const typename Tile<QT>::Lane lanes(lane, row_bytes);
    uint8_t* slot = slots + wave * Tile<QT>::kSlot;
    const int items = active ? (a.groups - ks + a.splits - 1) / a.splits : 0;   // (splits <= groups)
    Tile<QT> buf[kDepth];
    // (past the last item: it again)
    auto load = [&](auto slot_c, int j) __attribute__((always_inline)) {
        buf[decltype(slot_c)::value].load(w, lanes, uint32_t(ks + a.splits * max(0, min(j, items - 1))) * group_step,
                                          tile_bytes);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    static_assert(kDepth == 2, "the loop below names the slots");
    load(S0{}, 0);
    load(S1{}, 1);
    if (wave < a.groups) stage_token<QT>(staged + wave * unit_bytes<QT>(), 0, 1, x0, lane);
    for (int g = wave + kWaves; g < a.groups; g += kWaves)
        stage_token<QT>(staged + g * unit_bytes<QT>(), 0, 1, group_x(g), lane);
    lds_barrier();
    float acc = 0.f;
    const LaneTokens<QT> lt(lane, 0, 1);
    auto compute = [&](auto slot_c, int j) __attribute__((always_inline)) {
        const int g = ks + a.splits * j;
        const uint32_t start =
            whole_chunks<QT>() ? 0u : a.off + ((uint32_t(n) * row_bytes + uint32_t(g) * group_step) & 15u);
        // (one wave's LDS operations complete in order: the reads see these writes, and the next
        // writes come after the reads)
        buf[decltype(slot_c)::value].store(slot, lane, lanes);
        __builtin_amdgcn_wave_barrier();
        Group<QT> d;
        decode(d, slot + n * Tile<QT>::kRow, start, q, g, blocks, a.stride);
        acc = group_dot<QT>(d, staged + g * unit_bytes<QT>(), lt, acc);
        __builtin_amdgcn_wave_barrier();
    };
    for (int j = 0; j < items; j += 2) {
        compute(S0{}, j);
        load(S0{}, j + 2);
        if (j + 1 < items) compute(S1{}, j + 1);
        load(S1{}, j + 3);
    }
    if (q == 0) red[wave * 16 + n] = acc;
    lds_barrier();
    if (tid < tiles_wg * 16) {
        const int r = tid & 15, wt = tid >> 4;
        const int row = 16 * (blockIdx.x * tiles_wg + wt) + r;
        if (row < a.rows) {
            float v[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float* p = red + (2 * wt + m) * a.splits * 16 + r;
                v[m] = p[0];
                for (int k = 1; k < a.splits; ++k) v[m] += p[16 * k];
            }
            a.out[int64_t(blockIdx.y) * a.rows + row] = activate(v[0], a.act) * v[1];
        }
    }
}

// blockIdx.x: one 16-row tile of Y.  Wave w takes part w % splits of the groups of choices w / splits,
// w / splits + waves / splits, ..., and stages their h itself, a group at a time, in LDS of its own (no
// workgroup barrier until the end).  Every (choice, part) leaves its sum in LDS; a choice's parts are
// added in order, weighted, and the choices in order.
constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / 64;
constexpr int kOneTables = 16 + 3 * 4 * kMoeOneTopk;
template <int QT>
__global__ __launch_bounds__(kOneThreads) void moe_one_down_kernel(MoeArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int* valid_lds = reinterpret_cast<int*>(smem);
    int* list = reinterpret_cast<int*>(smem + 16);   // the choices that are this layer's,
    int* expert_of = list + kMoeOneTopk;             // their experts
    float* weight_of = reinterpret_cast<float*>(expert_of + kMoeOneTopk);           // and weights
    float* res = reinterpret_cast<float*>(smem + kOneTables);                       // [entry of list][part][16 rows]
    uint8_t* mine = reinterpret_cast<uint8_t*>(res + a.topk * a.splits * 16);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, q = lane >> 4;
    uint8_t* staged = mine + wave * (unit_bytes<QT>() + Tile<QT>::kSlot);
    uint8_t* slot = staged + unit_bytes<QT>();
    if (wave == 0) {   // (kMoeOneTopk lanes)
        const int e = lane < a.topk ? a.ids[lane] : -1;
        const float weight = lane < a.topk ? a.wts[lane] : 0.f;
        const bool ok = unsigned(e) < unsigned(a.experts);
        const unsigned long long m = __ballot(ok);
        if (ok) {
            const int at = __popcll(m & ((1ull << lane) - 1));
            list[at] = lane;
            expert_of[at] = e;
            weight_of[at] = weight;
        }
        if (lane == 0) *valid_lds = __popcll(m);
    }
    lds_barrier();
    const int valid = __builtin_amdgcn_readfirstlane(*valid_lds);
    const int tile = blockIdx.x;
    const int ks = wave % a.splits, first = wave / a.splits, step_of = kOneWaves / a.splits;
    const int per = (a.groups - ks + a.splits - 1) / a.splits;   // (splits <= groups)
    const int items = first < valid ? per * ((valid - first + step_of - 1) / step_of) : 0;
    const int blocks = row_blocks<QT>(a.in);
    const uint32_t row_bytes = uint32_t(a.row_bytes), tile_bytes = 16 * row_bytes;
    const uint32_t group_step = uint32_t(row_blocks_per_group<QT>() * a.stride);
    const typename Tile<QT>::Lane lanes(lane, row_bytes);
    struct Cursor {
        int at, i;   // choice list[at], item i of its groups
    };
    auto step = [&](Cursor& c) {
        if (++c.i == per) {
            c.i = 0;
            c.at += step_of;
        }
    };
    Tile<QT> buf[kDepth];
    float4 xs[kDepth];
    Cursor ld = {first, 0}, cp = ld;
    // (past the last item: the last one again)
    auto load = [&](auto slot_c) __attribute__((always_inline)) {
        constexpr int S = decltype(slot_c)::value;
        const int g = ks + a.splits * ld.i;
        const int e = __builtin_amdgcn_readfirstlane(expert_of[ld.at]);
        const int choice = __builtin_amdgcn_readfirstlane(list[ld.at]);
        const int k0 = 256 * g + 4 * lane;
        xs[S] = float4{0.f, 0.f, 0.f, 0.f};
        if (k0 < a.in) xs[S] = *reinterpret_cast<const float4*>(a.x + int64_t(choice) * a.in + k0);
        buf[S].load(a.w0 + (int64_t(e) * a.rows + 16 * tile) * a.row_bytes, lanes, uint32_t(g) * group_step, tile_bytes);
        Cursor next = ld;
        step(next);
        if (next.at < valid) ld = next;
    };
    float acc = 0.f;
    const LaneTokens<QT> lt(lane, 0, 1);
    auto compute = [&](auto slot_c) __attribute__((always_inline)) {
        constexpr int S = decltype(slot_c)::value;
        // (one wave's LDS operations complete in order: the reads below see these writes, and the
        // next group's writes come after them)
        stage_token<QT>(staged, 0, 1, xs[S], lane);
        buf[S].store(slot, lane, lanes);
        __builtin_amdgcn_wave_barrier();
        const int g = ks + a.splits * cp.i;
        const uint32_t start =
            whole_chunks<QT>() ? 0u : a.off + ((uint32_t(n) * row_bytes + uint32_t(g) * group_step) & 15u);
        Group<QT> w;
        decode(w, slot + n * Tile<QT>::kRow, start, q, g, blocks, a.stride);
        acc = group_dot<QT>(w, staged, lt, acc);
        __builtin_amdgcn_wave_barrier();
        if (cp.i == per - 1) {
            if (q == 0) res[(cp.at * a.splits + ks) * 16 + n] = acc;
            acc = 0.f;
        }
        step(cp);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    static_assert(kDepth == 2, "the loop below names the slots");
    if (items > 0) {
        load(S0{});
        load(S1{});
        for (int j = 0; j < items; j += 2) {
            compute(S0{});
            load(S0{});
            if (j + 1 < items) compute(S1{});
            load(S1{});
        }
    }
    lds_barrier();
    // a choice's parts (a thread per choice and row), then the choices of a row
    if (tid < 16 * valid) {   // (16 kMoeOneTopk <= kOneThreads)
        float* p = res + (tid >> 4) * a.splits * 16 + (tid & 15);
        float s = p[0];
        for (int k = 1; k < a.splits; ++k) s += p[16 * k];
        p[0] = s;
    }
    lds_barrier();
    if (tid < 16) {
        const int64_t at = 16 * tile + tid;
        const float before = a.residual ? a.residual[at] : 0.f;
        float y = 0.f;
#pragma unroll 4
        for (int v = 0; v < valid; ++v) y = fmaf(weight_of[v], res[v * a.splits * 16 + tid], y);
        a.out[at] = before + y;
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
    constexpr int kBatch = 4;   // rows in flight
    for (int j0 = 0; j0 < topk; j0 += kBatch) {
        float4 v[kBatch];
        bool live[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int64_t p = int64_t(m) * topk + min(j0 + i, topk - 1);
            live[i] = j0 + i < topk && unsigned(ids[p]) < unsigned(experts);
            v[i] = reinterpret_cast<const float4*>(rows_of + p * K)[c];   // (anything where nothing was written)
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (live[i]) {
                s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w;
            }
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

void set_layout(MoeArgs& a, int type, BlockLayout lay) {
    a.stride = lay.stride;
    a.off = lay.off;
    a.row_bytes = int64_t(a.in / block_values_of(type)) * lay.stride;
    a.groups = (a.in + 255) / 256;
}

// Largest power of two that is at most `v` (v >= 1).
int pow2_floor(int64_t v) {
    int p = 1;
    while (2 * p <= v) p *= 2;
    return p;
}

template <int QT, bool UP>
hipError_t launch_many(MoeArgs a, hipStream_t s) {
    // Tokens of a slot: four, or as many as fit in the LDS of a CU: four of rows of up to 35 (Q8_0) to 41 (Q4_K)
    // groups, one of the longest.
    constexpr size_t kFixed = kManyFixed + size_t(kWaves) * Tile<QT>::kSlot;
    static_assert(kFixed + 128 * size_t(unit_bytes<QT>()) <= kGfx950LdsBytes, "a token of the longest rows fits");
    const size_t per_token = size_t(a.groups) * unit_bytes<QT>();
    a.set = int(std::min<size_t>({4, (kGfx950LdsBytes - kFixed) / per_token, size_t(a.pairs)}));
    const int slots = std::min(a.pairs, a.experts + a.pairs / a.set);
    // units of 32 KiB of weights or more per wave: enough to outlast the staging, and short enough
    // that the last round of workgroups costs little; fewer while there are not two workgroups per CU
    // (64 experts of 2048 x 1024, k = 8, Q4_K: two tokens 30.0 -> 21.9 us, four 38.9 -> 32.3, eight 51.4 -> 48.8; one or
    // four per CU instead: eight 51.3 and 48.3, twelve 63.7 and 63.1 against 59.5)
    const int units = a.rows / 16 * (UP ? 2 : 1);
    const int64_t filled = int64_t(units) * slots / (kWaves * 512);
    const int per_wave = int(std::max<int64_t>(1, std::min<int64_t>(filled, 32768 / (16 * a.row_bytes))));
    const int grid = std::max(1, units / (kWaves * per_wave));
    hipLaunchKernelGGL((moe_many_kernel<QT, UP>), dim3(grid, slots), dim3(kThreads), kFixed + size_t(a.set) * per_token,
                       s, a);
    return hipGetLastError();
}

template <int QT>
hipError_t launch_one_up(MoeArgs a, hipStream_t s) {
    constexpr size_t kFixed = kWaves * 64 + size_t(kWaves) * Tile<QT>::kSlot;
    static_assert(kFixed + 128 * size_t(unit_bytes<QT>()) <= kGfx950LdsBytes, "the longest token fits");
    // A tile's groups over as many waves as fill the chip (about kOneUpWaves).
    const int tiles = a.rows / 16;
    const int64_t want = kOneUpWaves / std::max<int64_t>(1, int64_t(tiles) * 2 * a.topk);
    a.splits = pow2_floor(std::max<int64_t>(1, std::min<int64_t>({want, kWaves / 2, a.groups})));
    const int tiles_wg = kWaves / (2 * a.splits);
    hipLaunchKernelGGL((moe_one_up_kernel<QT>), dim3((tiles + tiles_wg - 1) / tiles_wg, a.topk), dim3(kThreads),
                       kFixed + size_t(a.groups) * unit_bytes<QT>(), s, a);
    return hipGetLastError();
}

template <int QT>
hipError_t launch_one_down(MoeArgs a, hipStream_t s) {
    a.splits = pow2_floor(std::max<int64_t>(1, std::min<int64_t>({kOneWaves / a.topk, kOneWaves, a.groups})));
    const size_t lds = kOneTables + size_t(a.topk) * a.splits * 64 +
                       size_t(kOneWaves) * (unit_bytes<QT>() + Tile<QT>::kSlot);
    hipLaunchKernelGGL((moe_one_down_kernel<QT>), dim3(a.rows / 16), dim3(kOneThreads), lds, s, a);
    return hipGetLastError();
}

#define MQ_MOE_INSTANCES(QT)                                     \
    template __global__ void moe_one_up_kernel<QT>(MoeArgs);     \
    template __global__ void moe_one_down_kernel<QT>(MoeArgs);   \
    template __global__ void moe_many_kernel<QT, true>(MoeArgs); \
    template __global__ void moe_many_kernel<QT, false>(MoeArgs);
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

size_t moe_scratch_bytes(int64_t M, int64_t topk, int64_t F, int64_t K) {
    // one token: h of every choice; more: its two factors for every pair, and the weighted rows
    if (moe_one(M, topk)) return h_bytes(topk, F);
    return h_bytes(2 * M * topk, F) + round_up256(size_t(M * topk) * size_t(K) * 4);
}

hipError_t moe_set_attributes(size_t lds_limit) {
    const int room = int(std::min(lds_limit, kGfx950LdsBytes));
    hipError_t e = hipSuccess;
    for (int type : {kQ4_0, kQ4_1, kQ5_0, kQ5_1, kQ8_0, kQ4_K, kQ5_K, kQ6_K})
        e = e != hipSuccess ? e : with_type(type, [&](auto qt) {
            constexpr int QT = decltype(qt)::value;
            const void* const kernels[] = {reinterpret_cast<const void*>(&moe_one_up_kernel<QT>),
                                           reinterpret_cast<const void*>(&moe_one_down_kernel<QT>),
                                           reinterpret_cast<const void*>(&moe_many_kernel<QT, true>),
                                           reinterpret_cast<const void*>(&moe_many_kernel<QT, false>)};
            hipError_t r = hipSuccess;
            for (const void* k : kernels)
                if (r == hipSuccess) r = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, room);
            return r;
        });
    return e;
}

hipError_t launch_moe_ffn(const MoeLayer& l, hipStream_t s, const char** name) {
    const int64_t pairs = l.M * l.topk;
    const bool one = moe_one(l.M, l.topk);
    float* h = static_cast<float*>(l.scratch);
    float* rows = reinterpret_cast<float*>(static_cast<uint8_t*>(l.scratch) + h_bytes(2 * pairs, l.F));
    *name = one ? "moe_one" : "moe_many";
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
    set_layout(a, l.gu_type, l.gu_layout);
    hipError_t e = with_type(l.gu_type, [&](auto qt) {
        constexpr int QT = decltype(qt)::value;
        return one ? launch_one_up<QT>(a, s) : launch_many<QT, true>(a, s);
    });
    if (e != hipSuccess) return e;
    a.w0 = l.Wd;
    a.w1 = nullptr;
    a.x = h;
    a.in = int(l.F);
    a.rows = int(l.K);
    a.residual = l.residual;
    a.out = one ? l.Y : rows;
    set_layout(a, l.d_type, l.d_layout);
    e = with_type(l.d_type, [&](auto qt) {
        constexpr int QT = decltype(qt)::value;
        return one ? launch_one_down<QT>(a, s) : launch_many<QT, false>(a, s);
    });
    if (one || e != hipSuccess) return e;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned(l.K) / 4 + 255) / 256, unsigned(l.M)), dim3(256), 0, s, rows,
                       l.ids, l.residual, l.Y, int(l.topk), int(l.E), int(l.K));
    return hipGetLastError();
}

}  // namespace mq
