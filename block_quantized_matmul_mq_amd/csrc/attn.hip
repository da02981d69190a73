// mq_attn: attention over the paged cache of keys and values in blocks of 4 or 8 bits.
//
//   O[t][h] = sum_j softmax_j(scale Q[t][h] . K[j]) V[j],  head h reads the cache's head h / (q_heads / heads),
//   over the keys j that token t sees; a token that sees none gets zeros.
//
// One pass over the keys with the running maximum and sum of the softmax, 32 keys a step, both products on
// the f16 matrix units at f32 accuracy (a factor of f32 as the sum of two f16, 22 bits; codes are exact):
//
//   S^T = K Q^T  v_mfma_f32_16x16x32_f16, A = 16 keys x 32 dimensions of one block, B = 16 query rows.  Two codes
//     become two f16 by an AND with an OR (1024 + code, or 1024 + 16 code where they lie four bits higher) and a packed
//     addition that takes 1024 and the offset off; the factor 16 is taken back in Q's copy for those dimensions.
//     (Left as the subnormals that the bits are without the OR, codes would cost half of that, but the matrix units
//     align their sums by the exponent field: scores then err by 2^-19.)  A block's sum gets the block's scale of its
//     key (f16 in the cache, v_fma_mix) on the way to the score.
//   O^T = V^T P^T  the same instruction, A = 16 dimensions x 32 keys, B = 16 rows' weights.  The accumulator
//     layout of S^T (lane l: row l % 16, keys 4 (l / 16) + i) is the operand layout of P^T for the key order in
//     which the cache keeps V, so the weights stay in their lane.  V's scale differs by key, the summed index: the
//     weight is multiplied by it, once per block of 32 dimensions, and split into two f16 then, in units of
//     2^-E that keep it in f16's upper range (E follows the largest scale so far).
//
// Queries: the G = q_heads / heads query heads of a cache head and the tokens of a sequence are one list of rows
// (token G + head), so that a decoded token uses the cache once for all its heads.  Two kernels:
//   attn_few   16 rows to a workgroup, whose four waves divide the keys: bound by the cache's bytes, which go from
//              memory to the lanes that use them, the next step's in flight; or, few workgroups, by one step's latency.
//   attn_many  128 rows to a workgroup (64 in dimensions above 128), a wave 32 (16) of them, over the same keys: bound by the vector unit, so the codes
//              are unpacked once for the workgroup, into LDS as operands; and V with its scale, as two f16 (exact:
//              f16 times a code), which takes the weights' multiplication and split per block off the waves for a third
//              matrix instruction.
// Both cut the keys of a tile into pieces over workgroups where there are few tiles, joined by the last one.
//
// Measured, 4 bits, heads of 128: one sequence of 32768 keys, 28 heads on 4, 24 us (0.8 TB/s; its pieces alone 15, the join of
// 64 pieces the rest); 64 sequences of up to 8192 keys, 40 heads on 8, 111 us (2.8 TB/s; of 8192 each 3.8 TB/s, a copy here
// reads and writes 4.7).  512 tokens over 8192 keys, 28 heads on 4: 200 us, 291 TF of the formula's operations, 2.5 times as many
// on the matrix units for f32 accuracy; these are busy 28 % of the time, the vector ALU 30 %.
//
// What is not finite: a NaN goes with the sum of weights, through pieces and their join; scores past f32's range, infinite scales of
// keys and large ones of values have paths of their own (raise and exponents; attend; Piece).
#include <algorithm>

#include "kv_layout.h"
#include "mmq_splitk.h"
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;                // keys of a step
constexpr int kCounters = 65536;         // of the scratch; cut tiles are at most kTarget
constexpr int kTarget = 512;             // workgroups that a call is cut into where it has fewer tiles (attn_few: half of it, or twice, see plan)
constexpr int kFewTiles = 768;           // tiles of 16 rows up to which attn_few takes sequences of any number of rows
constexpr int kMaxSplits = 64;
constexpr int kJoinRows = 4096;          // of attn_many: pieces times rows of a tile at most (LDS of the join)
constexpr int kMinManySteps = 8, kPieceSteps = 2;   // steps of a piece at least, and what its start and end cost
constexpr size_t kMaxSlots = 60 << 20;   // bytes of all pieces at most
// attn_many's weights are in units of 2^-kManyUnit, f16's normal range from 2^-20 on, and up to 2^kManySlack
constexpr float kManyUnit = 6.0f;
constexpr int kManySlack = 8;

struct AttnArgs {
    KvView c;
    const float* q;
    float* out;
    unsigned* counters;
    float* partial;
    int64_t q_stride;
    int T, q_heads, dim, group, causal, window, max_q, max_kv;
    int tiles, splits, chunk_steps;      // row tiles of a sequence, pieces of a tile's keys, steps of a piece
    float scale;
};

template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const u4 x = *reinterpret_cast<const u4*>(p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i + j] = x[j];
        }
    } else {
        static_assert(N == 2, "dwords of a lane");
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[0] = x.x;
        v[1] = x.y;
    }
}

__device__ __forceinline__ float half_of(uint32_t v, int i) {
    return static_cast<float>(__builtin_bit_cast(h2, v)[i]);
}

// op over the four lanes of a row (l, l ^ 16, l ^ 32, l ^ 48)
template <class Op>
__device__ __forceinline__ float row_all(float v, const Op& op) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto x = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t x0 = x[0], x1 = x[1];     // (a bit cast of x[1] itself reads element 0)
    v = op(__builtin_bit_cast(float, x0), __builtin_bit_cast(float, x1));
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto y = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const uint32_t y0 = y[0], y1 = y[1];
    return op(__builtin_bit_cast(float, y0), __builtin_bit_cast(float, y1));
}
__device__ __forceinline__ float row_max(float v) {
    return row_all(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float row_sum(float v) {
    return row_all(v, [](float a, float b) { return a + b; });
}

// The maximum of a row that has seen no key; of one whose scores all lie below f32's range it is kLowest.
constexpr float kNone = -__builtin_inff(), kLowest = -3.4028234663852886e38f;
// A row whose largest score passes f32's range, to either side: its weights are not known.  (Beside a score in range one
// below it weighs nothing.)
__device__ __forceinline__ bool out_of_range(float m) { return m != kNone && !(fabsf(m) < -kLowest); }

typedef float f2 __attribute__((ext_vector_type(2)));

// Two products p d (d f16) as f16 pairs, hi + lo to 22 bits: hi the rounded product, lo the rounded rest of the exact one.  Each is
// one instruction a value (v_fma_mixlo_f16, v_fma_mixhi_f16), as long as hi's sum with 0 is not taken away.  The empty asm
// keeps hi one value: formed a second time for the rest, in another way, it would round differently once in some
// thousand values and the sum miss by 2^-11.
__device__ __forceinline__ void split(f2 p, _Float16 d0, _Float16 d1, uint32_t& hi, uint32_t& lo) {
    const h2 a = {static_cast<_Float16>(fmaf(p[0], static_cast<float>(d0), 0.0f)),
                  static_cast<_Float16>(fmaf(p[1], static_cast<float>(d1), 0.0f))};
    hi = __builtin_bit_cast(uint32_t, a);
    asm("" : "+v"(hi));
    const h2 h = __builtin_bit_cast(h2, hi);
    const h2 b = {static_cast<_Float16>(fmaf(p[0], static_cast<float>(d0), -static_cast<float>(h[0]))),
                  static_cast<_Float16>(fmaf(p[1], static_cast<float>(d1), -static_cast<float>(h[1])))};
    lo = __builtin_bit_cast(uint32_t, b);
}
// The same of two f32 values.  one: 1, in a register (as a constant it would cost the rest a conversion more).
__device__ __forceinline__ void split(f2 w, float one, uint32_t& hi, uint32_t& lo) {
    hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, h2));
    asm("" : "+v"(hi));
    const h2 h = __builtin_bit_cast(h2, hi);
    const h2 b = {static_cast<_Float16>(fmaf(w[0], one, -static_cast<float>(h[0]))),
                  static_cast<_Float16>(fmaf(w[1], one, -static_cast<float>(h[1])))};
    lo = __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ float opaque_one() {
    float one = 1.0f;
    asm("" : "+v"(one));
    return one;
}

// The bits of two codes in a dword, in registers of the vector unit: its AND-OR takes one scalar operand only.
struct Masks {
    uint32_t low, up;
    template <int BITS>
    static __device__ __forceinline__ Masks make() {
        Masks m = {BITS == 8 ? 0x00FF00FFu : 0x000F000Fu, 0x00F000F0u};
        asm("" : "+v"(m.low), "+v"(m.up));
        return m;
    }
};

// The keys and values of one step as they lie in the cache: two tiles of 16 tokens.
template <int BITS, int D>
struct Step {
    static constexpr int kDwords = D * BITS / 128;      // code dwords of a lane and tile, K or V
    static constexpr int kScales = D / 16;              // scale dwords: 4 tokens of D / 32
    uint32_t k[2][kDwords], v[2][kDwords], ks[2][kScales], vs[2][kScales];
    bool there[2];                                      // (uniform) the tile has a page

    __device__ __forceinline__ void load(const KvView& c, const int (&pages)[2], int head, int key0, int lane) {
        using L = KvLayout<BITS, D>;
        const int64_t section = int64_t(c.page_tokens) * L::kRow;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            there[t] = pages[t] >= 0;
            const int slot = (key0 + 16 * t) & (c.page_tokens - 1);
            const uint8_t* p = c.data + (int64_t(max(pages[t], 0)) * c.heads + head) * c.chunk;
            load_dwords(p + slot * L::kRow + (lane & 15) * L::kRow + (lane >> 4) * (L::kRow / 4), k[t]);
            load_dwords(p + section + slot * L::kRow + lane * (L::kRow / 4), v[t]);
            const uint8_t* s = p + 2 * section + (slot + 4 * (lane >> 4)) * (2 * L::kBlocks);
            load_dwords(s, ks[t]);
            load_dwords(s + int64_t(c.page_tokens) * (2 * L::kBlocks), vs[t]);
        }
    }
};

// A wave's 16 query rows: operands, running statistics and sums.
template <int BITS, int D>
struct Rows {
    static constexpr int kBlocks = D / 32;
    static constexpr int kTiles = D / 16;
    h8 hi[kBlocks], lo[kBlocks];
    f4 o[kTiles];
    float f;                        // score in log2 units per unit of the accumulated sums
    float m, l;                     // the score (log2 units) that weights are relative to, or none; this lane's part of the sum of weights
    float least;                    // attn_few: the least score seen (unscaled, or 0)
    bool far;                       // (uniform) a row's m is far (see exponents)
    int first, last;                // keys first .. last - 1 are seen

    // q: the row's f32 values, of which this lane has 8 in each block
    __device__ __forceinline__ void init(const float* q, float scale, int lane) {
        const int g = lane >> 4;
        float x[kBlocks][8];
        float top = 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f4 v = *reinterpret_cast<const f4*>(q + 32 * b + 8 * g + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[b][4 * i + j] = scale < 0.0f ? -v[j] : v[j];
                    top = fmaxf(top, fabsf(v[j]));
                }
            }
        }
        top = row_max(top);
        // q 2^a: the row's largest value just under 2^14 (f16 ends at 2^16; what falls below its normal range is
        // then 2^-28 of the largest)
        int e = 0;
        if (top > 0.0f && top <= 3.4028235e38f) e = 14 - (ilogbf(top) + 1);
        // (half of log2 e, so that the product holds for every scale; not 0: a masked score times f stays -inf; and finite)
        f = fminf(fmaxf(ldexpf(fabsf(scale) * 0.721347520444481703f, 1 - e), 0x1p-126f), -kLowest);
        constexpr int kOrder4[8] = {0, 4, 1, 5, 2, 6, 3, 7}, kOrder8[8] = {0, 2, 1, 3, 4, 6, 5, 7};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            u4 h, l;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                f2 v;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    v[j] = ldexpf(x[b][BITS == 4 ? kOrder4[i + j] : kOrder8[i + j]], BITS == 4 && (i & 2) ? e - 4 : e);   // (codes 16 times as large)
                uint32_t u, w;
                split(v, 1.0f, u, w);
                h[i / 2] = u;
                l[i / 2] = w;
            }
            hi[b] = __builtin_bit_cast(h8, h);
            lo[b] = __builtin_bit_cast(h8, l);
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[j] = f4{0, 0, 0, 0};
        m = kNone;
        far = false;
        l = least = 0.0f;
    }
    // The score that weights are relative to follows these scores' maximum where that passes it by more than SLACK (a weight
    // may so be up to 2^SLACK, and the sums are rescaled in few steps only).  It is a rounded product, but the same in every
    // weight's exponent, so that its rounding drops out as long as f16 has room for it (see exponents).
    template <int SLACK>
    __device__ __forceinline__ float raise(const float (&sc)[8]) {
        float top = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
        top = row_max(top);
        const bool up = fmaf(top, f, -m) > float(SLACK);      // (no score seen, none before: NaN, no)
        if (__ballot(up) != 0) {
            const float to = up ? fmaxf(top * f, kLowest) : m;
            const float keep = !up || m == kNone ? 1.0f : __builtin_amdgcn_exp2f(m - to);
            l *= keep;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) o[j] *= keep;
            m = to;
            far = __ballot(m != kNone && is_far(m)) != 0;
        }
        return m == kNone ? 0.0f : m;
    }
    // Weight i is exp2(sc[i] by - base), 2^unit for a score of top (raise's).  Usually by = f, in one fma.  The roundings of top and
    // base shift all weights of the row by up to 2^(1/2) below 2^23, which f16 has room for, but by 2^8 and more from 2^27 on: from
    // 2^23 on scores are rounded to f32 (as they would be in a matrix of scores) before top is taken off.  any_far: a row of
    // the wave is there.
    static __device__ __forceinline__ bool is_far(float top) { return fabsf(top) >= 0x1p23f; }
    template <int SLACK>
    __device__ __forceinline__ void exponents(float (&sc)[8], float top, float unit, bool any_far, float& by, float& base) const {
#pragma clang fp contract(off)
        by = f;
        base = top - unit;
        if (any_far) {
            const bool mine = is_far(top);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = sc[i] * f - top;          // (the exact difference is SLACK at most)
                sc[i] = mine ? (d > float(SLACK) ? float(SLACK) : d) : sc[i];
            }
            by = mine ? 1.0f : f;
            base = mine ? -unit : base;
        }
    }
};

// Two codes from where the mask finds them in the dword, offset taken off: 1024 + code as f16, less 1024 + offset; of codes
// that lie four bits up, 16 times the code less 16 times the offset.
template <int BITS>
__device__ __forceinline__ uint32_t two_codes(const Masks& m, uint32_t w, bool up) {
    const _Float16 off = static_cast<_Float16>(BITS == 8 || up ? -1152.0f : -1032.0f);
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (w & (up ? m.up : m.low)) | 0x64006400u) + h2{off, off});
}

// The codes of K's block b as a matrix operand.
template <int BITS, int N>
__device__ __forceinline__ h8 key_codes(const Masks& m, const uint32_t (&k)[N], int b) {
    u4 a;
    if constexpr (BITS == 4) {
        const uint32_t w = k[b], x = w >> 8;
        a = u4{two_codes<4>(m, w, false), two_codes<4>(m, w, true), two_codes<4>(m, x, false), two_codes<4>(m, x, true)};
    } else {
        const uint32_t w = k[2 * b], x = k[2 * b + 1];
        a = u4{two_codes<8>(m, w, false), two_codes<8>(m, w >> 8, false), two_codes<8>(m, x, false), two_codes<8>(m, x >> 8, false)};
    }
    return __builtin_bit_cast(h8, a);
}

// Codes of V's dimensions 16 j .. 16 j + 15 (of which this lane supplies one) for the step's 32 keys; for 4 bits and odd
// j, 16 times the codes.
template <int BITS, int D>
__device__ __forceinline__ h8 value_codes(const Masks& m, const Step<BITS, D>& s, int j) {
    constexpr int kPer = BITS == 4 ? 4 : 2;                 // 16s of dimensions in a unit
    constexpr int kUnits = KvLayout<BITS, D>::kUnits;
    const int i = j / kPer, n = j % kPer;
    u4 a;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t w = s.v[p >> 1][(p & 1) * kUnits + i];
        if (BITS == 8 ? n == 1 : n >= 2) w >>= 8;
        a[p] = two_codes<BITS>(m, w, BITS == 4 && (n & 1));
    }
    return __builtin_bit_cast(h8, a);
}

// One step for one set of rows.  full: every row sees every key.
template <int BITS, int D>
__device__ __forceinline__ void attend(const Masks& masks, const Step<BITS, D>& s, Rows<BITS, D>& r, int key0, bool full, int lane, float unit_e) {
    constexpr int kBlocks = D / 32;
    // (all blocks' first products, then their second ones: neither waits for another)
    float sc[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        f4 acc[kBlocks];
        h8 k[kBlocks];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            k[b] = key_codes<BITS>(masks, s.k[t], b);
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[b], r.hi[b], f4{0, 0, 0, 0}, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[b], r.lo[b], acc[b], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[4 * t + i] = 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sc[4 * t + i] = fmaf(half_of(s.ks[t][i * (kBlocks / 2) + b / 2], b & 1), acc[b][i], sc[4 * t + i]);
    }
    // (The sums of finite operands stay below 2^48: a score of -inf comes from a scale that is an infinity, and would pass for a key
    // that is not seen.  The kernel's end makes the row NaN.  Four v_min3 a step: 64 sequences of up to 8192 keys 110.2 -> 111.6 us.)
    uint32_t seen = 0xFF;
    if (!full) {
        seen = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int key = key0 + 16 * (i >> 2) + 4 * (lane >> 4) + (i & 3);
            const bool ok = key >= r.first && key < r.last && s.there[i >> 2];
            r.least = ok ? fminf(r.least, sc[i]) : r.least;
            sc[i] = ok ? sc[i] : kNone;
            seen |= uint32_t(ok) << i;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) r.least = fminf(fminf(r.least, sc[i]), sc[i + 1]);
    }
    float by, base, p[8];
    const float top = r.template raise<4>(sc);
    r.template exponents<4>(sc, top, unit_e, r.far, by, base);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], by, -base));
        r.l += p[i];
    }
    // V's scales, 0 of keys that the row does not see (whose bits may be anything)
    uint32_t vs[8][kBlocks / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int b = 0; b < kBlocks / 2; ++b) vs[i][b] = s.vs[i >> 2][(i & 3) * (kBlocks / 2) + b];
    if (!full) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int b = 0; b < kBlocks / 2; ++b) vs[i][b] = seen >> i & 1 ? vs[i][b] : 0;
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        u4 h, l;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            uint32_t u, w;
            split(f2{p[i], p[i + 1]}, __builtin_bit_cast(h2, vs[i][b / 2])[b & 1], __builtin_bit_cast(h2, vs[i + 1][b / 2])[b & 1], u, w);
            h[i / 2] = u;
            l[i / 2] = w;
        }
        const h8 hi = __builtin_bit_cast(h8, h), lo = __builtin_bit_cast(h8, l);
        const h8 a0 = value_codes<BITS, D>(masks, s, 2 * b), a1 = value_codes<BITS, D>(masks, s, 2 * b + 1);
        r.o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, hi, r.o[2 * b], 0, 0, 0);
        r.o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, hi, r.o[2 * b + 1], 0, 0, 0);
        r.o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a0, lo, r.o[2 * b], 0, 0, 0);
        r.o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a1, lo, r.o[2 * b + 1], 0, 0, 0);
    }
}

// The largest magnitude of V's scales in this lane, a NaN where one is.
template <int BITS, int D>
__device__ __forceinline__ float scale_top(const Step<BITS, D>& s) {
    auto at = [&](int i) { return __builtin_bit_cast(h2, s.vs[i / Step<BITS, D>::kScales][i % Step<BITS, D>::kScales]); };
    h2 hi = at(0), lo = hi;
#pragma unroll
    for (int i = 1; i + 1 < 2 * Step<BITS, D>::kScales; i += 2) {      // (two a time: v_pk_maximum3_f16)
        hi = __builtin_elementwise_maximum(__builtin_elementwise_maximum(hi, at(i)), at(i + 1));
        lo = __builtin_elementwise_minimum(__builtin_elementwise_minimum(lo, at(i)), at(i + 1));
    }
    hi = __builtin_elementwise_maximum(hi, at(2 * Step<BITS, D>::kScales - 1));
    lo = __builtin_elementwise_minimum(lo, at(2 * Step<BITS, D>::kScales - 1));
    hi = __builtin_elementwise_maximum(hi, -lo);
    return __builtin_elementwise_maximum(static_cast<float>(hi[0]), static_cast<float>(hi[1]));
}
// The largest exponent field of the finite scales of the keys that the lane's row sees in the step.
template <int BITS, int D>
__device__ __forceinline__ int scale_exponent(const Step<BITS, D>& s, int key0, int first, int last, int lane) {
    int top = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < Step<BITS, D>::kScales; ++i) {
            const int key = key0 + 16 * t + 4 * (lane >> 4) + i / (D / 64);
            const int a = (s.vs[t][i] >> 10) & 31, b = (s.vs[t][i] >> 26) & 31;
            if (key >= first && key < last && s.there[t]) top = max(top, max(a == 31 ? 0 : a, b == 31 ? 0 : b));
        }
#pragma unroll
    for (int off = 32; off >= 16; off >>= 1) top = max(top, __shfl_xor(top, off, 64));
    return top;
}

// A workgroup's part of the call: a tile of rows of one cache head, and of a piece of its keys.
struct Work {
    int head, seq, tile, split, cell;
    int q0, n, rows, row0;           // the sequence's first row, its rows, rows of the list, this tile's first
    int past, len;                   // the first row's position in the cache; cached tokens as far as they count
};
__device__ __forceinline__ int wrapping(unsigned a, unsigned b) { return int(a + b); }
__device__ __forceinline__ bool work_of(const AttnArgs& a, int tile_rows, Work& w) {
    // heads vary fastest (workgroups are dealt to the XCDs in turn, whose L2 so holds few heads); later rows, which
    // see more keys, come first, and a tile's last piece, which is rarely a whole one, comes last
    int item = blockIdx.x;
    w.head = item % a.c.heads;
    item /= a.c.heads;
    w.seq = item % a.c.seqs;
    item /= a.c.seqs;
    w.tile = a.tiles - 1 - item % a.tiles;
    w.split = item / a.tiles;
    w.cell = (w.seq * a.tiles + w.tile) * a.c.heads + w.head;
    w.q0 = a.c.q_start[w.seq];
    // (rows inside the call's whatever the arrays hold, and sums that may wrap without a sign: starts of any value make a product
    // n group that wraps to rows that are not there)
    const int all = wrapping(a.c.q_start[w.seq + 1], -unsigned(w.q0));
    w.n = w.q0 < 0 ? 0 : max(0, min(all, min(a.max_q, a.T - w.q0)));
    w.rows = w.n * a.group;
    w.row0 = w.tile * tile_rows;
    const int real = a.c.kv_len[w.seq];
    w.past = wrapping(real, -unsigned(all));
    w.len = min(real, a.max_kv);
    return w.row0 < w.rows;
}
// Keys [first, last) that a token of the sequence sees.
__device__ __forceinline__ int first_key(const AttnArgs& a, const Work& w, int tok) {
    return a.window > 0 ? max(0, wrapping(w.past, tok + 1 - a.window)) : 0;
}
__device__ __forceinline__ int last_key(const AttnArgs& a, const Work& w, int tok) {
    return a.causal ? min(w.len, wrapping(w.past, tok + 1)) : w.len;
}
__device__ __forceinline__ const float* query_row(const AttnArgs& a, const Work& w, int row) {
    const int tok = row / a.group;
    return a.q + int64_t(w.q0 + tok) * a.q_stride + int64_t(w.head * a.group + row - tok * a.group) * (a.dim);
}
__device__ __forceinline__ float* out_row(const AttnArgs& a, const Work& w, int row) {
    const int tok = row / a.group;
    return a.out + (int64_t(w.q0 + tok) * a.q_heads + w.head * a.group + row - tok * a.group) * a.dim;
}
__device__ __forceinline__ void pages_of(const AttnArgs& a, const Work& w, int step, int (&pages)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) pages[t] = __builtin_amdgcn_readfirstlane(kv_page(a.c, w.seq, step * kStep + 16 * t));
}

// A piece's rows to its slot of the scratch (sums, then maxima in log2 units, then sums of weights).
template <int D, int ROWS>
struct Slot {
    static constexpr int kFloats = ROWS * (D + 2);
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ Slot(const AttnArgs& a, int cell) {
        rsrc = __builtin_amdgcn_make_buffer_rsrc(a.partial + int64_t(cell) * a.splits * kFloats, 0, a.splits * kFloats * 4,
                                                 0x00020000);
    }
    __device__ __forceinline__ void put(int split, int row, const f4 (&o)[D / 16], float m, float l, int lane) const {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(splitk_u4, o[j]), rsrc,
                                                   (row * D + 16 * j + 4 * (lane >> 4)) * 4, split * kFloats * 4, kSplitkSc1);
        if (lane < 16) {
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, m), rsrc, (ROWS * D + row) * 4,
                                                  split * kFloats * 4, kSplitkSc1);
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, l), rsrc, (ROWS * (D + 1) + row) * 4,
                                                  split * kFloats * 4, kSplitkSc1);
        }
    }
    // The last piece: every row's sums, in the order of the pieces.  share: LDS of pieces * ROWS floats.
    __device__ __forceinline__ void join(const AttnArgs& a, const Work& w, int pieces, float* share) const {
        const int live = min(ROWS, w.rows - w.row0);
        auto word = [&](int piece, int at) {
            return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, at * 4, piece * kFloats * 4, kSplitkSc1));
        };
        // A thread's first sums, and kTeam threads a row, each the statistics of some of its pieces: all of these loads in flight
        // together (a trip to the device-coherent level is more than a microsecond).
        constexpr int kFirst = ROWS == 16 && D <= 128 ? 16 : 8, kItems = D / 4;
        constexpr int kTeam = kThreads / ROWS;
        auto sums = [&](int piece, int item) {
            return __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, item * 16, piece * kFloats * 4, kSplitkSc1));
        };
        f4 ahead[kFirst];
        const int mine = min(int(threadIdx.x), live * kItems - 1);
#pragma unroll
        for (int p = 0; p < kFirst; ++p) ahead[p] = sums(min(p, pieces - 1), mine);
        const int row_of = threadIdx.x / kTeam, sub = threadIdx.x % kTeam;
        if (row_of < live) {
            float top = kNone, sum = 0.0f;
            for (int p = sub; p < pieces; p += kTeam) {
                const float m = word(p, ROWS * D + row_of), l = word(p, ROWS * (D + 1) + row_of);
                share[p * ROWS + row_of] = m;
                // (sums so far follow a larger maximum; a piece without one has a sum of 0, or of NaN where its scores are NaN)
                const float to = fmaxf(top, m);
                sum = fmaf(sum, top == kNone ? 1.0f : __builtin_amdgcn_exp2f(top - to), m == kNone ? l : l * __builtin_amdgcn_exp2f(m - to));
                top = to;
            }
            float all = top;
#pragma unroll
            for (int off = kTeam / 2; off; off >>= 1) all = fmaxf(all, __shfl_xor(all, off, 64));
            sum = top == kNone ? sum : sum * __builtin_amdgcn_exp2f(top - all);
            // (the team's sums in a fixed order: the result is the same every time)
#pragma unroll
            for (int off = kTeam / 2; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
            const float inv = out_of_range(all) ? __builtin_nanf("") : sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int p = sub; p < pieces; p += kTeam) {
                float& s = share[p * ROWS + row_of];
                s = s == kNone ? (inv == inv ? 0.0f : inv) : __builtin_amdgcn_exp2f(s - all) * inv;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < live * kItems; i += kThreads) {
            const int row = i / kItems;
            f4 sum = {0, 0, 0, 0};
            int p = 0;
            auto add = [&](const f4& v, int piece) {
                const float x = share[piece * ROWS + row];
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[j], x, sum[j]);
            };
            if (i == int(threadIdx.x)) {
#pragma unroll
                for (int k = 0; k < kFirst; ++k)
                    if (k < pieces) add(ahead[k], k);
                p = min(kFirst, pieces);
            }
            auto batch = [&](auto n_c) {      // that many loads in flight
                constexpr int kN = decltype(n_c)::value;
                for (; p + kN <= pieces; p += kN) {
                    f4 v[kN];
#pragma unroll
                    for (int k = 0; k < kN; ++k) v[k] = sums(p + k, i);
#pragma unroll
                    for (int k = 0; k < kN; ++k) add(v[k], p + k);
                }
            };
            if constexpr (ROWS == 16 && D <= 128) batch(std::integral_constant<int, 24>{});
            batch(std::integral_constant<int, 16>{});
            batch(std::integral_constant<int, 8>{});
            batch(std::integral_constant<int, 4>{});
            batch(std::integral_constant<int, 2>{});
            batch(std::integral_constant<int, 1>{});
            *reinterpret_cast<f4*>(out_row(a, w, w.row0 + row) + i % kItems * 4) = sum;
        }
    }
};

template <int D>
__device__ __forceinline__ void write_row(float* out, const f4 (&o)[D / 16], float m, float l, int lane) {
    const float inv = out_of_range(m) ? __builtin_nanf("") : l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) *reinterpret_cast<f4*>(out + 16 * j + 4 * (lane >> 4)) = o[j] * inv;
}

// 16 rows; the waves take steps in turn.
template <int BITS, int D>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void attn_few_kernel(AttnArgs a) {
    constexpr int kTiles = D / 16, kRows = 16;
    constexpr int kPad = 4;                                  // (rows a bank apart)
    __shared__ float part[2][kRows][D + kPad];
    __shared__ float stat[kWaves][2][kRows];
    __shared__ float share[kMaxSplits * kRows];
    __shared__ unsigned ticket;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Work w;
    if (!work_of(a, kRows, w)) return;
    const int tok0 = w.row0 / a.group, tok1 = (min(w.row0 + kRows, w.rows) - 1) / a.group;
    const int begin = first_key(a, w, tok0) / kStep, end = (max(0, last_key(a, w, tok1)) + kStep - 1) / kStep;   // steps
    const int full_begin = first_key(a, w, tok1), full_end = last_key(a, w, tok0);   // keys that every row sees
    const int pieces = max(1, (end - begin + a.chunk_steps - 1) / a.chunk_steps);
    if (w.split >= pieces) return;
    const int from = begin + w.split * a.chunk_steps, to = min(end, from + a.chunk_steps);
    Rows<BITS, D> r;
    const int row = min(w.row0 + (lane & 15), w.rows - 1);
    r.init(query_row(a, w, row), a.scale, lane);
    r.first = first_key(a, w, row / a.group);
    r.last = last_key(a, w, row / a.group);
    // Weights are kept in units of 2^-unit_e, so that they stay in f16's upper range times V's scales: the largest scale
    // seen (2^(x - 14) at most, x its exponent field) is 2^7 then; a weight to 2^4 and a scale 2^4 times as large fit
    // before the units change.  A row has its own: what it does not see may not take bits from what it sees.
    constexpr int kRoom = 21;
    int unit_e = 0;
    float unit_top = -1.0f;          // scales to this fit
    const Masks masks = Masks::make<BITS>();
    auto take = [&](const Step<BITS, D>& s, int step) {
        const int key0 = step * kStep;
        if (__ballot(!(scale_top(s) <= unit_top)) != 0) {
            const int x = scale_exponent(s, key0, r.first, r.last, lane);
            if (unit_top < 0.0f || x > kRoom - unit_e + 4) {
                const float by = ldexpf(1.0f, kRoom - x - unit_e);
                r.l *= by;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) r.o[j] *= by;
                unit_e = kRoom - x;
                unit_top = ldexpf(1.0f, x - 14 + 4);
            }
        }
        const bool full = key0 >= full_begin && key0 + kStep <= full_end && s.there[0] && s.there[1];
        attend<BITS, D>(masks, s, r, key0, full, lane, float(unit_e));
    };
    // A step's loads are in flight while the one before is worked on, its page numbers one step earlier.  Behind the
    // last step the last one is read again: loads without a branch, so that the wait for a step leaves the next one's be.
    int step = from + wave;
    if (step < to) {
        auto at = [&](int n) { return min(step + n * kWaves, to - 1); };
        Step<BITS, D> s;
        int pages[2];
        pages_of(a, w, step, pages);
        s.load(a.c, pages, w.head, step * kStep, lane);
        pages_of(a, w, at(1), pages);
        if constexpr (D > 128) {      // (heads of 256: two steps' loads do not fit the registers)
            for (;;) {
                take(s, step);
                step += kWaves;
                if (step >= to) break;
                s.load(a.c, pages, w.head, step * kStep, lane);
                pages_of(a, w, at(1), pages);
            }
        } else for (Step<BITS, D> t;;) {
            t.load(a.c, pages, w.head, at(1) * kStep, lane);
            pages_of(a, w, at(2), pages);
            take(s, step);
            step += kWaves;
            if (step >= to) break;
            s.load(a.c, pages, w.head, at(1) * kStep, lane);
            pages_of(a, w, at(2), pages);
            take(t, step);
            step += kWaves;
            if (step >= to) break;
        }
    }
    const float back = ldexpf(1.0f, -unit_e);
    if (r.least == kNone) r.l = __builtin_nanf("");
    r.l = row_sum(r.l) * back;
#pragma unroll
    for (int j = 0; j < kTiles; ++j) r.o[j] *= BITS == 4 && (j & 1) ? back * 0.0625f : back;
    // the waves' sums relative to the largest of their maxima, added in pairs through LDS
    if (lane < 16) {
        stat[wave][0][lane] = r.m;
        stat[wave][1][lane] = r.l;
    }
    __syncthreads();
    {
        const int c = lane & 15;
        float top = kNone, sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) top = fmaxf(top, stat[v][0][c]);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
            const float m = stat[v][0][c];
            sum = fmaf(stat[v][1][c], m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - top), sum);
        }
        const float keep = r.m == kNone ? 0.0f : __builtin_amdgcn_exp2f(r.m - top);
#pragma unroll
        for (int j = 0; j < kTiles; ++j) r.o[j] = r.m == kNone ? f4{0, 0, 0, 0} : r.o[j] * keep;
        r.m = top;
        r.l = sum;
    }
    static_assert(kWaves == 4, "pairs");
    for (int stage = 2; stage >= 1; stage >>= 1) {
        if (wave >= stage && wave < 2 * stage)
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
                *reinterpret_cast<f4*>(&part[wave - stage][lane & 15][16 * j + 4 * (lane >> 4)]) = r.o[j];
        __syncthreads();
        if (wave < stage)
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
                r.o[j] += *reinterpret_cast<const f4*>(&part[wave][lane & 15][16 * j + 4 * (lane >> 4)]);
        __syncthreads();
    }
    const bool live = w.row0 + (lane & 15) < w.rows;
    if (pieces == 1) {
        if (wave == 0 && live) write_row<D>(out_row(a, w, row), r.o, r.m, r.l, lane);
        return;
    }
    const Slot<D, kRows> slot(a, w.cell);
    if (wave == 0 && live) slot.put(w.split, lane & 15, r.o, r.m, r.l, lane);
    if (!splitk_arrive(a.counters + w.cell, pieces, &ticket)) return;
    slot.join(a, w, pieces, share);
}

// Four waves, each with 16 RT rows; the workgroup's steps go through LDS as operands, two buffers.
template <int BITS, int D>
struct Staged {
    static constexpr int kBlocks = D / 32, kTiles = D / 16;
    u4 k[2][kBlocks][64];            // [16 keys][block][lane]
    u4 v_hi[kTiles][64], v_lo[kTiles][64];
    float ks[2][kBlocks][16];        // K's scales
    uint32_t vs[2][kBlocks * 8];     // V's, as in the cache: [16 tokens][block]
    uint32_t special[kWaves], bad[kWaves], large[kWaves];   // per wave, of V's scales: see Piece::stage
};

// What a thread loads of a step and lays into LDS: K's codes of some blocks of a lane; V's units of a lane and of two tokens,
// with these tokens' scales; the first threads a dword of both kinds of scales.
template <int BITS, int D>
struct Piece {
    using L = KvLayout<BITS, D>;
    static constexpr int kBlocks = D / 32, kUnits = L::kUnits;
    static constexpr int kOps = kBlocks / 2;               // of K's 128 (lane, tile) times kBlocks operands
    static constexpr int kDs = BITS == 4 ? kUnits : kUnits / 2;
    static constexpr int kScaleDwords = kBlocks * 16;      // of K, or V, of a step
    static_assert(kThreads == 256 && kScaleDwords <= kThreads, "one piece a thread");
    uint32_t k[kOps * BITS / 4], v[kUnits], d[2 * kDs], ks, vs;

    template <int N>
    static __device__ __forceinline__ void load_any(const uint8_t* p, uint32_t* v) {
        if constexpr (N >= 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<u4*>(v + i) = *reinterpret_cast<const u4*>(p + 4 * i);
        } else if constexpr (N == 2) {
            *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        } else {
            *v = *reinterpret_cast<const uint32_t*>(p);
        }
    }
    __device__ __forceinline__ void load(const KvView& c, const int (&pages)[2], int head, int key0) {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int section = c.page_tokens * L::kRow;
        const uint8_t* base[2];
        int slot[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            base[t] = c.data + (int64_t(max(pages[t], 0)) * c.heads + head) * c.chunk;
            slot[t] = (key0 + 16 * t) & (c.page_tokens - 1);
        }
        const int kt = wave / 2, h = wave % 2;
        load_any<kOps * BITS / 4>((kt ? base[1] : base[0]) + (kt ? slot[1] : slot[0]) * L::kRow + (lane & 15) * L::kRow +
                                      (lane >> 4) * (L::kRow / 4) + h * (kOps * BITS), k);
        const int vt = (tid >> 1) & 1, pair = tid & 1, ln = tid >> 2;
        const uint8_t* p = (vt ? base[1] : base[0]) + section;
        const int s = vt ? slot[1] : slot[0];
        load_any<kUnits>(p + s * L::kRow + ln * (L::kRow / 4) + pair * kUnits * 4, v);
        const uint8_t* q = p + section + (c.page_tokens + s + 4 * (ln >> 4) + 2 * pair) * (2 * kBlocks);
        load_any<kDs>(q, d);
        load_any<kDs>(q + 2 * kBlocks, d + kDs);
        if (tid < kScaleDwords) {
            const int t = tid / (kBlocks * 8), o = tid % (kBlocks * 8);
            const uint8_t* p = (t ? base[1] : base[0]) + 2 * section + (t ? slot[1] : slot[0]) * (2 * kBlocks) + 4 * o;
            ks = *reinterpret_cast<const uint32_t*>(p);
            vs = *reinterpret_cast<const uint32_t*>(p + c.page_tokens * (2 * kBlocks));
        }
    }
    // V's scale times a code (for 4 bits and odd 16s of dimensions 16 times the code) is held as two f16, exactly, as long as the
    // products stay below f16's end: scales under 2^8 (times 128).  The quick form says in `special` where a scale is an infinity, a
    // NaN or larger; its products of that step are then made again in the ordinary form, which takes those as 0 and says in `bad`
    // where one is not finite, in `large` where a finite one is larger.  The products of large ones alone, times kSmall, are the
    // third form, for a product of their own: rows that do not see them, and smaller values beside them, lose nothing.
    enum Form { kQuick, kOrdinary, kLargeOnes };
    static constexpr int kLarge = 23;                       // exponent field
    static constexpr float kSmall = 0x1p-8f;
    template <Form FORM>
    __device__ __forceinline__ void stage(const Masks& masks, Staged<BITS, D>& s, const int (&pages)[2], int key0, int len) const {
        const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        if constexpr (FORM != kLargeOnes)
#pragma unroll
            for (int b = 0; b < kOps; ++b) s.k[wave / 2][wave % 2 * kOps + b][lane] = __builtin_bit_cast(u4, key_codes<BITS>(masks, k, b));
        bool special = false, bad = false, large = false;
        const int t = (tid >> 1) & 1, pair = tid & 1, ln = tid >> 2;
        uint32_t e[2 * kDs];             // the scales, 0 behind the sequence's end
#pragma unroll
        for (int i = 0; i < 2 * kDs; ++i) e[i] = d[i];
        if (key0 + kStep > len || pages[0] < 0 || pages[1] < 0) {
            const int key = key0 + 16 * t + 4 * (ln >> 4) + 2 * pair;
            const bool there = (t ? pages[1] : pages[0]) >= 0;
#pragma unroll
            for (int i = 0; i < 2 * kDs; ++i) e[i] = there && key + i / kDs < len ? e[i] : 0;
        }
        if constexpr (FORM == kQuick) {
            typedef unsigned short us2 __attribute__((ext_vector_type(2)));
            us2 top = {0, 0};
#pragma unroll
            for (int i = 0; i < 2 * kDs; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(us2, e[i] & 0x7FFF7FFFu));
            special = top[0] >= (kLarge << 10) || top[1] >= (kLarge << 10);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * kDs; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = (e[i] >> (16 * h + 10)) & 31;
                    const bool is_large = x >= kLarge && x < 31;
                    bad |= x == 31;
                    large |= is_large;
                    if (FORM == kOrdinary ? x >= kLarge : !is_large) e[i] &= h ? 0x0000FFFFu : 0xFFFF0000u;
                }
        }
        uint32_t* hi = reinterpret_cast<uint32_t*>(s.v_hi);
        uint32_t* lo = reinterpret_cast<uint32_t*>(s.v_lo);
        constexpr int kPer = BITS == 4 ? 4 : 2;         // 16s of dimensions in a unit
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
            for (int n = 0; n < kPer; ++n) {
                // the two tokens' scales of the unit's block
                const int word = BITS == 4 ? i : i / 2;
                const bool second = BITS == 4 ? n >= 2 : (i & 1) != 0;
                const h2 dd = __builtin_bit_cast(h2, __builtin_amdgcn_perm(e[kDs + word], e[word], second ? 0x07060302u : 0x05040100u));
                uint32_t x = v[i];
                if (BITS == 8 ? n == 1 : n >= 2) x >>= 8;
                const h2 c = __builtin_bit_cast(h2, two_codes<BITS>(masks, x, BITS == 4 && (n & 1)));
                uint32_t h, l;
                if constexpr (FORM == kQuick) {
                    const h2 p = c * dd;
                    h = __builtin_bit_cast(uint32_t, p);
                    l = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(c, dd, -p));
                } else {
                    const float by = FORM == kLargeOnes ? kSmall : 1.0f;
                    split(f2{static_cast<float>(c[0]) * (static_cast<float>(dd[0]) * by),
                             static_cast<float>(c[1]) * (static_cast<float>(dd[1]) * by)}, 1.0f, h, l);
                }
                const int at = ((i * kPer + n) * 64 + ln) * 4 + (tid & 3);
                hi[at] = h;
                lo[at] = l;
            }
        if constexpr (FORM == kLargeOnes) return;
        const bool any_special = __ballot(special) != 0, any_bad = __ballot(bad) != 0, any_large = __ballot(large) != 0;
        if (lane == 0) {
            s.special[wave] = any_special;
            s.bad[wave] = any_bad;
            s.large[wave] = any_large;
        }
        if (tid < kScaleDwords) {
            const int tt = tid / (kBlocks * 8), o = tid % (kBlocks * 8), token = o / (kBlocks / 2), b = 2 * (o % (kBlocks / 2));
            // (an infinity as a NaN: a score of -inf would pass for a key that is not seen)
            s.ks[tt][b][token] = fmaf(half_of(ks, 0), 0.0f, half_of(ks, 0));
            s.ks[tt][b + 1][token] = fmaf(half_of(ks, 1), 0.0f, half_of(ks, 1));
            s.vs[tt][o] = vs;
        }
    }
};

template <int N>
__device__ __forceinline__ bool any_of(const uint32_t (&v)[N]) {
    uint32_t all = v[0];
#pragma unroll
    for (int i = 1; i < N; ++i) all |= v[i];
    return __builtin_amdgcn_readfirstlane(all) != 0;
}

// One staged step for a wave's RT sets of rows.  large: V's products of large scales (Piece::stage), or null.
template <int BITS, int D, int RT>
__device__ __forceinline__ void attend_staged(const Staged<BITS, D>& s, const Staged<BITS, D>* large, Rows<BITS, D> (&r)[RT], int key0,
                                              bool full, bool there0, bool there1, int lane) {
    constexpr int kBlocks = D / 32, kTiles = D / 16;
    // Operands are read from LDS one product ahead (the scheduling barriers keep it at that: all of them at once take more
    // registers than there are), and a block's sums are used while the next block's products run.
    float sc[RT][8];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[i][j] = 0.0f;
    u4 k = s.k[0][0][lane];
    f4 d = *reinterpret_cast<const f4*>(&s.ks[0][0][4 * (lane >> 4)]), d1;
    f4 acc[RT], acc1[RT];
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int n = 0; n <= 2 * kBlocks; ++n) {
        const int b = n % kBlocks, tn = (n + 1) / kBlocks % 2, bn = (n + 1) % kBlocks;
        const h8 k0 = __builtin_bit_cast(h8, k);
        const f4 d0 = d;
        if (n + 1 < 2 * kBlocks) {
            k = s.k[tn][bn][lane];
            d = *reinterpret_cast<const f4*>(&s.ks[tn][bn][4 * (lane >> 4)]);
        }
        if (n < 2 * kBlocks) {
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, r[i].hi[b], f4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, r[i].lo[b], acc[i], 0, 0, 0);
        }
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float& x = sc[i][4 * ((n - 1) / kBlocks) + j];
                    x = (n - 1) % kBlocks == 0 ? d1[j] * acc1[i][j] : fmaf(d1[j], acc1[i][j], x);
                }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) acc1[i] = acc[i];
        d1 = d0;
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    // (One code path with the masks as a branch over a few selects; the asm keeps the scores here, whose sums the compiler
    // otherwise moves behind the branches of another row set, holding every operand until then.)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) asm volatile("" : "+v"(sc[i][j]));
    if (!full) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = key0 + 16 * (j >> 2) + 4 * (lane >> 4) + (j & 3);
                sc[i][j] = key >= r[i].first && key < r[i].last && (j < 4 ? there0 : there1) ? sc[i][j] : kNone;
            }
    }
    const float one = opaque_one();
    h8 hi[RT], lo[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        float by, base;
        const float top = r[i].template raise<kManySlack>(sc[i]);
        // (asked at each step: kept over the steps, as in attn_few, it is slower here: 512 tokens over 8192 keys 201 -> 204 us)
        r[i].template exponents<kManySlack>(sc[i], top, kManyUnit, __ballot(Rows<BITS, D>::is_far(top)) != 0, by, base);
        u4 h, l;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            f2 p;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                p[k] = __builtin_amdgcn_exp2f(fmaf(sc[i][j + k], by, -base));
                r[i].l += p[k];
            }
            uint32_t u, w;
            split(p, one, u, w);
            h[j / 2] = u;
            l[j / 2] = w;
        }
        hi[i] = __builtin_bit_cast(h8, h);
        lo[i] = __builtin_bit_cast(h8, l);
    }
    __builtin_amdgcn_s_setprio(1);
    u4 vh[2], vl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        vh[k] = s.v_hi[k][lane];
        vl[k] = s.v_lo[k][lane];
    }
#pragma unroll
    for (int j = 0; j < kTiles; j += 2) {
        h8 h[2], l[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            h[k] = __builtin_bit_cast(h8, vh[k]);
            l[k] = __builtin_bit_cast(h8, vl[k]);
            if (j + 2 < kTiles) {
                vh[k] = s.v_hi[j + 2 + k][lane];
                vl[k] = s.v_lo[j + 2 + k][lane];
            }
        }
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    r[i].o[j + k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(m < 2 ? h[k] : l[k], m == 1 ? lo[i] : hi[i], r[i].o[j + k], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    if (large) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            const h8 h = __builtin_bit_cast(h8, large->v_hi[j][lane]), l = __builtin_bit_cast(h8, large->v_lo[j][lane]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                f4 sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(h, hi[i], f4{0, 0, 0, 0}, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(h, lo[i], sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(l, hi[i], sum, 0, 0, 0);
                r[i].o[j] += sum * (1.0f / Piece<BITS, D>::kSmall);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

template <int BITS, int D>
__global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void attn_many_kernel(AttnArgs a) {
    constexpr int RT = D <= 128 ? 2 : 1, kTiles = D / 16, kBlocks = D / 32, kRows = 16 * kWaves * RT;
    constexpr size_t kBuffers = 2 * sizeof(Staged<BITS, D>), kJoin = kJoinRows * sizeof(float);
    __shared__ __align__(16) uint8_t memory[kBuffers > kJoin ? kBuffers : kJoin];
    __shared__ unsigned ticket;
    Staged<BITS, D>* const buf = reinterpret_cast<Staged<BITS, D>*>(memory);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Work w;
    if (!work_of(a, kRows, w)) return;
    const int tok0 = w.row0 / a.group, tok1 = (min(w.row0 + kRows, w.rows) - 1) / a.group;
    const int begin = first_key(a, w, tok0) / kStep, end = (max(0, last_key(a, w, tok1)) + kStep - 1) / kStep;   // steps
    const int pieces = max(1, (end - begin + a.chunk_steps - 1) / a.chunk_steps);
    if (w.split >= pieces) return;
    const int from = begin + w.split * a.chunk_steps, to = min(end, from + a.chunk_steps);
    // the wave's own rows, and the keys that every one of them sees
    const int mine = w.row0 + wave * 16 * RT;
    const int t0 = min(mine, w.rows - 1) / a.group, t1 = (min(mine + 16 * RT, w.rows) - 1) / a.group;
    const int full_begin = first_key(a, w, t1), full_end = last_key(a, w, t0);
    Rows<BITS, D> r[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = min(mine + 16 * i + (lane & 15), w.rows - 1);
        r[i].init(query_row(a, w, row), a.scale, lane);
        r[i].first = first_key(a, w, row / a.group);
        r[i].last = last_key(a, w, row / a.group);
    }
    using P = Piece<BITS, D>;
    if (from < to) {
        const Masks masks = Masks::make<BITS>();
        P piece;
        int pages[2], next[2];
        pages_of(a, w, from, pages);
        piece.load(a.c, pages, w.head, from * kStep);
        piece.template stage<P::kQuick>(masks, buf[0], pages, from * kStep, w.len);
        pages_of(a, w, min(from + 1, to - 1), next);
        __syncthreads();
        for (int step = from; step < to; ++step) {
            const int key0 = step * kStep;
            Staged<BITS, D>&s = buf[(step - from) & 1], &t = buf[(step + 1 - from) & 1];
            bool large = false;
            if (any_of(s.special)) {         // (the piece is still this step's, and the other buffer free)
                __syncthreads();
                piece.template stage<P::kOrdinary>(masks, s, pages, key0, w.len);
                __syncthreads();
                large = any_of(s.large);
                if (large) {
                    piece.template stage<P::kLargeOnes>(masks, t, pages, key0, w.len);
                    __syncthreads();
                }
            }
            const bool there0 = pages[0] >= 0, there1 = pages[1] >= 0;
            const int ahead = min(step + 1, to - 1);
            pages[0] = next[0];
            pages[1] = next[1];
            piece.load(a.c, pages, w.head, ahead * kStep);
            pages_of(a, w, min(step + 2, to - 1), next);
            const bool full = key0 >= full_begin && key0 + kStep <= full_end && there0 && there1;
            attend_staged<BITS, D, RT>(s, large ? &t : nullptr, r, key0, full, there0, there1, lane);
            if (any_of(s.bad)) {      // (staged as zeros)
                for (int i = 0; i < kStep; ++i)
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        const uint32_t d = s.vs[i >> 4][(i & 15) * (kBlocks / 2) + b / 2] >> (16 * (b & 1));
                        if ((d & 0x7C00u) != 0x7C00u) continue;
#pragma unroll
                        for (int k = 0; k < RT; ++k)
                            if (key0 + i >= r[k].first && key0 + i < r[k].last && (i < 16 ? there0 : there1)) {
                                const float nan = __builtin_nanf("");
                                r[k].o[2 * b] = r[k].o[2 * b + 1] = f4{nan, nan, nan, nan};
                            }
                    }
            }
            if (large) __syncthreads();      // (every wave is through with the other buffer)
            piece.template stage<P::kQuick>(masks, t, pages, ahead * kStep, w.len);
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        r[i].l = row_sum(r[i].l);
        if constexpr (BITS == 4)
#pragma unroll
            for (int j = 1; j < kTiles; j += 2) r[i].o[j] *= 0.0625f;
    }
    const Slot<D, kRows> slot(a, w.cell);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = mine + 16 * i + (lane & 15);
        if (row >= w.rows) continue;
        if (pieces == 1) write_row<D>(out_row(a, w, row), r[i].o, r[i].m, r[i].l, lane);
        else slot.put(w.split, row - w.row0, r[i].o, r[i].m, r[i].l, lane);
    }
    if (pieces == 1 || !splitk_arrive(a.counters + w.cell, pieces, &ticket)) return;
    slot.join(a, w, pieces, reinterpret_cast<float*>(memory));
}

// How a call is cut: into tiles of 16 rows, or of 128 (64 in dimensions above 128) where a sequence has more than 256 and tiles of 16
// would be more than kFewTiles; and the keys of a tile into pieces where there are few tiles.  Both sides, in us, 4-bit caches:
//   rows x sequences and heads, keys, dimension    attn_few  attn_many
//     84 x  4,  4096, 128                            17        51
//    259 x 24,  4096, 128                            83        91
//    511 x  4,  4096, 128                            31        63
//   1029 x  4,  4096, 128                            61        69
//    511 x 24,  4096, 128 (768 tiles of 16)         106       102     (the rule's loss: 4)
//   1029 x 24,  4096, 128                           228       195
//   2100 x 24,   600, 128                            80        58
//    511 x 96,   600, 128                            85        65
//    259 x 96,   600, 256                           150       121
//   2100 x  4,  4096, 128 (528 tiles)               102        88     (the rule's loss: 14)
struct Plan {
    int tile_rows, tiles, splits, chunk_steps;
    int64_t blocks;
};
size_t slot_bytes(int rows, int64_t dim) { return size_t(rows) * size_t(dim + 2) * 4; }
Plan plan(int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t max_q, int64_t max_kv) {
    Plan p;
    const int64_t rows = max_q * (q_heads / heads), steps = (max_kv + kStep - 1) / kStep + 1;
    p.tile_rows = rows <= 256 || seqs * heads * ((rows + 15) / 16) <= kFewTiles ? 16 : dim > 128 ? 64 : 128;
    const int64_t tiles = (rows + p.tile_rows - 1) / p.tile_rows, items = seqs * heads * tiles;
    int64_t splits = 1;
    if (p.tile_rows == 16) {
        // pieces of 8 steps for a workgroup per CU, of 64 steps for four (lengths differ: pieces even them out)
        const int64_t n = std::max(std::min(kTarget / 2 / items, steps / 8), std::min(2 * kTarget / items, steps / 64));
        splits = std::max<int64_t>(1, std::min<int64_t>(kMaxSplits, n));
    } else {
        // the number of pieces that keeps rounds of kTarget workgroups fullest, a piece's start and end at the price of kPieceSteps
        const int64_t most = std::min<int64_t>(kJoinRows / p.tile_rows, steps / kMinManySteps);
        double best = 0.0;
        for (int64_t n = 1; n == 1 || (n <= most && size_t(n * items) * slot_bytes(p.tile_rows, dim) <= kMaxSlots); ++n) {
            const int64_t chunk = (steps + n - 1) / n, blocks = items * n;
            const double full = double(blocks) / double((blocks + kTarget - 1) / kTarget * kTarget);
            const double rate = full * double(chunk) / double(chunk + kPieceSteps + (n > 1 ? 1 : 0));
            if (rate > best) {
                best = rate;
                splits = n;
            }
        }
    }
    p.chunk_steps = int((steps + splits - 1) / splits);
    p.splits = int((steps + p.chunk_steps - 1) / p.chunk_steps);
    p.tiles = int(tiles);
    p.blocks = items * p.splits;
    return p;
}

}  // namespace

size_t attn_scratch_bytes(int, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t max_q, int64_t max_kv) {
    const Plan p = plan(seqs, q_heads, heads, dim, max_q, max_kv);
    return size_t(kCounters) * 4 + (p.splits > 1 ? size_t(p.blocks) * slot_bytes(p.tile_rows, dim) : 0);
}

// (a grid's threads are counted in 32 bits)
bool attn_fits(int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t max_q, int64_t max_kv) {
    return plan(seqs, q_heads, heads, dim, max_q, max_kv).blocks * kThreads < (int64_t(1) << 32);
}

hipError_t launch_attn(const Attn& r, hipStream_t s, const char** name) {
    const Plan p = plan(r.cache.view.seqs, r.q_heads, r.cache.view.heads, r.cache.dim, r.max_q, r.max_kv);
    *name = p.tile_rows == 16 ? "attn_few" : "attn_many";
    AttnArgs a;
    a.c = r.cache.view;
    a.q = r.q;
    a.out = r.out;
    a.counters = static_cast<unsigned*>(r.scratch);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(r.scratch) + size_t(kCounters) * 4);
    a.q_stride = r.q_stride;
    a.T = int(r.T);
    a.q_heads = int(r.q_heads);
    a.dim = int(r.cache.dim);
    a.group = int(r.q_heads / r.cache.view.heads);
    a.causal = r.causal;
    a.window = int(r.window);
    a.max_q = int(r.max_q);
    a.max_kv = int(r.max_kv);
    a.tiles = p.tiles;
    a.splits = p.splits;
    a.chunk_steps = p.chunk_steps;
    a.scale = r.scale;
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(unsigned(p.blocks)), dim3(kThreads), 0, s, a); };
    kv_kinds(r.cache.bits, r.cache.dim, [&](auto bits, auto dim) {
        constexpr int kB = decltype(bits)::value, kD = decltype(dim)::value;
        if (p.tile_rows == 16) run(attn_few_kernel<kB, kD>);
        else run(attn_many_kernel<kB, kD>);
    });
    return hipGetLastError();
}

}  // namespace mq
