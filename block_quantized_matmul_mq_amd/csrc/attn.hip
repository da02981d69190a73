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
// (token G + head), cut into tiles of 16 RT rows per wave, so that a decoded token uses the cache once for all its heads.
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
constexpr int kTarget = 512;             // workgroups that a call is cut into where it has fewer tiles
constexpr int kMaxSplits = 128;
constexpr int kMinSteps = 4;             // steps of a wave at least where a tile's keys are cut

struct AttnArgs {
    KvView c;
    const float* q;
    float* out;
    unsigned* counters;
    float* partial;
    int64_t q_stride;
    int T, q_heads, group, causal, window, max_q, max_kv;
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

constexpr float kNone = -__builtin_inff();

typedef float f2 __attribute__((ext_vector_type(2)));

// Two values as f16 pairs, hi + lo to 22 bits: hi rounded from the f32 values w, lo from the exact rest p d - hi (w = p d
// rounded).  The empty asm keeps hi one value: formed a second time for the rest, by a fused instruction from the
// exact product, it would round the other way once in some thousand values and the sum miss by 2^-11.
__device__ __forceinline__ void split(f2 p, f2 d, uint32_t& hi, uint32_t& lo) {
    const f2 w = p * d;
    hi = __builtin_bit_cast(uint32_t, __builtin_convertvector(w, h2));
    asm("" : "+v"(hi));
    const h2 h = __builtin_bit_cast(h2, hi);
    const f2 rest = {fmaf(p[0], d[0], -static_cast<float>(h[0])), fmaf(p[1], d[1], -static_cast<float>(h[1]))};
    lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, h2));
}

// The keys and values of one step as they lie in the cache: two tiles of 16 tokens.
template <int BITS, int D>
struct Step {
    static constexpr int kDwords = D * BITS / 128;      // code dwords of a lane and tile, K or V
    static constexpr int kScales = D / 16;              // scale dwords: 4 tokens of D / 32
    uint32_t k[2][kDwords], v[2][kDwords], ks[2][kScales], vs[2][kScales];
    bool there[2];                                      // (uniform) the tile has a page

    __device__ __forceinline__ void load(const KvView& c, int seq, int head, int key0, int lane) {
        using L = KvLayout<BITS, D>;
        const int64_t section = int64_t(c.page_tokens) * L::kRow;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int key = key0 + 16 * t;
            int page = __builtin_amdgcn_readfirstlane(kv_page(c, seq, key));
            there[t] = page >= 0;
            page = there[t] ? page : 0;
            const int slot = key & (c.page_tokens - 1);
            const uint8_t* p = c.data + (int64_t(page) * c.heads + head) * c.chunk;
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
    float m, l;                     // the largest sum so far (or none), this lane's part of the sum of weights
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
        f = ldexpf(fabsf(scale) * 1.44269504088896341f, -e);
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
                split(v, f2{1.0f, 1.0f}, u, w);
                h[i / 2] = u;
                l[i / 2] = w;
            }
            hi[b] = __builtin_bit_cast(h8, h);
            lo[b] = __builtin_bit_cast(h8, l);
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[j] = f4{0, 0, 0, 0};
        m = kNone;
        l = 0.0f;
    }
};

// Two codes from where `mask` finds them in the dword, offset taken off: 1024 + code as f16, less 1024 + offset; of codes
// that lie four bits up, 16 times the code less 16 times the offset.
template <int BITS>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, bool up) {
    const uint32_t mask = BITS == 8 ? 0x00FF00FFu : up ? 0x00F000F0u : 0x000F000Fu;
    const _Float16 off = static_cast<_Float16>(BITS == 8 || up ? -1152.0f : -1032.0f);
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, (w & mask) | 0x64006400u) + h2{off, off});
}

// The codes of K's block b as a matrix operand.
template <int BITS, int N>
__device__ __forceinline__ h8 key_codes(const uint32_t (&k)[N], int b) {
    u4 a;
    if constexpr (BITS == 4) {
        const uint32_t w = k[b], x = w >> 8;
        a = u4{two_codes<4>(w, false), two_codes<4>(w, true), two_codes<4>(x, false), two_codes<4>(x, true)};
    } else {
        const uint32_t w = k[2 * b], x = k[2 * b + 1];
        a = u4{two_codes<8>(w, false), two_codes<8>(w >> 8, false), two_codes<8>(x, false), two_codes<8>(x >> 8, false)};
    }
    return __builtin_bit_cast(h8, a);
}

// Codes of V's dimensions 16 j .. 16 j + 15 (of which this lane supplies one) for the step's 32 keys; for 4 bits and odd
// j, 16 times the codes.
template <int BITS, int D>
__device__ __forceinline__ h8 value_codes(const Step<BITS, D>& s, int j) {
    constexpr int kPer = BITS == 4 ? 4 : 2;                 // 16s of dimensions in a unit
    constexpr int kUnits = KvLayout<BITS, D>::kUnits;
    const int i = j / kPer, n = j % kPer;
    u4 a;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t w = s.v[p >> 1][(p & 1) * kUnits + i];
        if (BITS == 8 ? n == 1 : n >= 2) w >>= 8;
        a[p] = two_codes<BITS>(w, BITS == 4 && (n & 1));
    }
    return __builtin_bit_cast(h8, a);
}

// One step for one set of rows.  MASKED: some row does not see some key.
template <int BITS, int D, bool MASKED>
__device__ __forceinline__ void attend(const Step<BITS, D>& s, Rows<BITS, D>& r, int key0, int lane, float unit) {
    constexpr int kBlocks = D / 32, kTiles = D / 16;
    float sc[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[4 * t + i] = 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const h8 a = key_codes<BITS>(s.k[t], b);
            f4 acc = {0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, r.hi[b], acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, r.lo[b], acc, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sc[4 * t + i] = fmaf(half_of(s.ks[t][i * (kBlocks / 2) + b / 2], b & 1), acc[i], sc[4 * t + i]);
        }
    }
    bool ok[8];
    if constexpr (MASKED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int key = key0 + 16 * (i >> 2) + 4 * (lane >> 4) + (i & 3);
            ok[i] = key >= r.first && key < r.last && s.there[i >> 2];
            sc[i] = ok[i] ? sc[i] : kNone;
        }
    }
    float top = fmaxf(fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3])), fmaxf(fmaxf(sc[4], sc[5]), fmaxf(sc[6], sc[7])));
    top = fmaxf(row_max(top), r.m);
    // weights relative to the stored (rounded) m f, so that its rounding drops out
    const float base = top == kNone ? 0.0f : top * r.f;
    if (__ballot(top != r.m) != 0) {
        const float keep = r.m == kNone ? 1.0f : __builtin_amdgcn_exp2f(r.m * r.f - base);
        r.l *= keep;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) r.o[j] *= keep;
        r.m = top;
    }
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], r.f, -base));
        if constexpr (MASKED) p[i] = ok[i] ? p[i] : 0.0f;
        r.l += p[i];
        p[i] *= unit;
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        u4 h, l;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            f2 d;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t v = s.vs[i >> 2][((i + j) & 3) * (kBlocks / 2) + b / 2];
                if constexpr (MASKED) v = ok[i + j] ? v : 0;
                d[j] = half_of(v, b & 1);
            }
            uint32_t u, w;
            split(f2{p[i], p[i + 1]}, d, u, w);
            h[i / 2] = u;
            l[i / 2] = w;
        }
        const h8 hi = __builtin_bit_cast(h8, h), lo = __builtin_bit_cast(h8, l);
#pragma unroll
        for (int j = 2 * b; j < 2 * b + 2; ++j) {
            const h8 a = value_codes<BITS, D>(s, j);
            r.o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, hi, r.o[j], 0, 0, 0);
            r.o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, lo, r.o[j], 0, 0, 0);
        }
    }
}

// A bound on the exponent field (f16) of V's scales of the step, the bits of all of them together: quick, and
// at most one less than a power of two.
template <int BITS, int D>
__device__ __forceinline__ int scale_bits(const Step<BITS, D>& s) {
    uint32_t all = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < Step<BITS, D>::kScales; ++i) all |= s.vs[t][i];
    all |= all >> 16;
    return (all >> 10) & 31;
}
// The largest exponent field of the finite scales of the sequence's tokens in the step; uniform.
template <int BITS, int D>
__device__ __forceinline__ int scale_exponent(const Step<BITS, D>& s, int key0, int len, int lane) {
    int top = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < Step<BITS, D>::kScales; ++i) {
            const int key = key0 + 16 * t + 4 * (lane >> 4) + i / (D / 64);
            const int a = (s.vs[t][i] >> 10) & 31, b = (s.vs[t][i] >> 26) & 31;
            if (key < len && s.there[t]) top = max(top, max(a == 31 ? 0 : a, b == 31 ? 0 : b));
        }
#pragma unroll
    for (int off = 32; off >= 16; off >>= 1) top = max(top, __shfl_xor(top, off, 64));
    return __builtin_amdgcn_readfirstlane(top);
}

// KW: waves that share their rows and divide the keys (4: few rows; 1: each wave has rows of its own).
template <int BITS, int D, int RT, int KW>
__global__ __launch_bounds__(kThreads) void attn_kernel(AttnArgs a) {
    constexpr int kTiles = D / 16;
    constexpr int kRows = 16 * RT;
    constexpr int kPad = 4;                                  // (rows a bank apart)
    __shared__ float part[KW > 1 ? 2 : 1][KW > 1 ? kRows : 1][KW > 1 ? D + kPad : 1];
    __shared__ float stat[KW > 1 ? KW : 1][2][KW > 1 ? kRows : 1];
    __shared__ float share[KW > 1 ? kMaxSplits : 1][KW > 1 ? kRows : 1];
    __shared__ unsigned ticket;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads vary fastest (workgroups are dealt to the XCDs in turn, whose L2 so holds few heads), later rows, which
    // see more keys, come first
    int item = blockIdx.x;
    const int head = item % a.c.heads;
    item /= a.c.heads;
    const int split = item % a.splits;
    item /= a.splits;
    const int tile = a.tiles - 1 - item % a.tiles, seq = item / a.tiles;
    const int q0 = a.c.q_start[seq], all = a.c.q_start[seq + 1] - q0;
    const int n = q0 < 0 ? 0 : min(all, min(a.max_q, a.T - q0));
    const int rows = n * a.group;
    const int row0 = (KW > 1 ? tile : tile * kWaves + wave) * kRows;
    if (row0 >= rows) return;                                // (KW > 1: the whole workgroup)
    const int real = a.c.kv_len[seq], len = min(real, a.max_kv);
    const int tok0 = row0 / a.group, tok1 = (min(row0 + kRows, rows) - 1) / a.group;
    // keys that some row of the tile sees, and keys that every row sees
    auto first_of = [&](int tok) { return a.window > 0 ? max(0, real - all + tok + 1 - a.window) : 0; };
    auto last_of = [&](int tok) { return a.causal ? min(len, real - all + tok + 1) : len; };
    const int begin = first_of(tok0) / kStep, end = (max(0, last_of(tok1)) + kStep - 1) / kStep;   // steps
    const int full_begin = first_of(tok1), full_end = last_of(tok0);
    int from = begin, to = end, pieces = 1;
    if constexpr (KW > 1) {
        pieces = max(1, (end - begin + a.chunk_steps - 1) / a.chunk_steps);
        if (split >= pieces) return;
        from = begin + split * a.chunk_steps;
        to = min(end, from + a.chunk_steps);
    }
    Rows<BITS, D> r[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = min(row0 + 16 * i + (lane & 15), rows - 1);
        const int tok = row / a.group, h = head * a.group + row - tok * a.group;
        r[i].init(a.q + int64_t(q0 + tok) * a.q_stride + int64_t(h) * D, a.scale, lane);
        r[i].first = first_of(tok);
        r[i].last = last_of(tok);
    }
    // Weights times scales are kept in units of 2^-unit_e: the largest scale seen (2^(x - 14) at most, x its exponent
    // field) is 2^7 then, so a later one may be 2^8 times as large before the units change.
    constexpr int kRoom = 21, kLimit = 29, kUnset = 1000;
    float unit = 1.0f;
    int unit_e = kUnset;
    Step<BITS, D> s;
    for (int step = from + (KW > 1 ? wave : 0); step < to; step += KW) {
        const int key0 = step * kStep;
        s.load(a.c, seq, head, key0, lane);
        if (__ballot(scale_bits(s) > kLimit - unit_e) != 0) {
            const int x = scale_exponent(s, key0, len, lane);
            if (x > kLimit - unit_e) {
                const float by = unit_e == kUnset ? 1.0f : ldexpf(1.0f, kRoom - x - unit_e);
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) r[i].o[j] *= by;
                unit_e = kRoom - x;
                unit = ldexpf(1.0f, unit_e);
            }
        }
        const bool full = key0 >= full_begin && key0 + kStep <= full_end && s.there[0] && s.there[1];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if (full) attend<BITS, D, false>(s, r[i], key0, lane, unit);
            else attend<BITS, D, true>(s, r[i], key0, lane, unit);
        }
    }
    const float back = 1.0f / unit;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        r[i].l = row_sum(r[i].l);
        r[i].m = r[i].m == kNone ? kNone : r[i].m * r[i].f;      // log2 units from here on
#pragma unroll
        for (int j = 0; j < kTiles; ++j) r[i].o[j] *= BITS == 4 && (j & 1) ? back * 0.0625f : back;
    }
    auto out_of = [&](int row) {
        const int tok = row / a.group, h = head * a.group + row - tok * a.group;
        return a.out + (int64_t(q0 + tok) * a.q_heads + h) * D;
    };
    if constexpr (KW == 1) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = row0 + 16 * i + (lane & 15);
            if (row >= rows) continue;
            const float inv = r[i].l == 0.0f ? 0.0f : 1.0f / r[i].l;
            float* out = out_of(row) + 4 * (lane >> 4);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) *reinterpret_cast<f4*>(out + 16 * j) = r[i].o[j] * inv;
        }
    } else {
        // the waves' sums relative to the largest of their maxima, added in pairs through LDS
#pragma unroll
        for (int i = 0; i < RT; ++i)
            if (lane < 16) {
                stat[wave][0][16 * i + lane] = r[i].m;
                stat[wave][1][16 * i + lane] = r[i].l;
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int row = 16 * i + (lane & 15);
            float top = kNone, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < KW; ++w) top = fmaxf(top, stat[w][0][row]);
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const float m = stat[w][0][row];
                sum = fmaf(stat[w][1][row], m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - top), sum);
            }
            const float keep = r[i].m == kNone ? 0.0f : __builtin_amdgcn_exp2f(r[i].m - top);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) r[i].o[j] = r[i].m == kNone ? f4{0, 0, 0, 0} : r[i].o[j] * keep;
            r[i].m = top;
            r[i].l = sum;
        }
        static_assert(KW == 4, "pairs");
        for (int stage = 2; stage >= 1; stage >>= 1) {
            if (wave >= stage && wave < 2 * stage)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
                        *reinterpret_cast<f4*>(&part[wave - stage][16 * i + (lane & 15)][16 * j + 4 * (lane >> 4)]) = r[i].o[j];
            __syncthreads();
            if (wave < stage)
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < kTiles; ++j)
                        r[i].o[j] += *reinterpret_cast<const f4*>(&part[wave][16 * i + (lane & 15)][16 * j + 4 * (lane >> 4)]);
            __syncthreads();
        }
        if (pieces == 1) {
            if (wave == 0)
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int row = row0 + 16 * i + (lane & 15);
                    if (row >= rows) continue;
                    const float inv = r[i].l == 0.0f ? 0.0f : 1.0f / r[i].l;
                    float* out = out_of(row) + 4 * (lane >> 4);
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) *reinterpret_cast<f4*>(out + 16 * j) = r[i].o[j] * inv;
                }
            return;
        }
        // a piece of the keys: its sums and statistics to its slot, the last piece joins them (mmq_splitk.h)
        constexpr int kSlot = kRows * (D + 2);               // floats: sums, then maxima, then sums of weights
        const int cell = (seq * a.tiles + tile) * a.c.heads + head;
        float* slots = a.partial + int64_t(cell) * a.splits * kSlot;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(slots, 0, a.splits * kSlot * 4, 0x00020000);
        const int live = min(kRows, rows - row0);
        if (wave == 0)
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int row = 16 * i + (lane & 15);
                if (row >= live) continue;
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(splitk_u4, r[i].o[j]), rsrc,
                                                           (row * D + 16 * j + 4 * (lane >> 4)) * 4, split * kSlot * 4, kSplitkSc1);
                if (lane < 16) {
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, r[i].m), rsrc, (kRows * D + row) * 4,
                                                          split * kSlot * 4, kSplitkSc1);
                    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, r[i].l), rsrc, (kRows * (D + 1) + row) * 4,
                                                          split * kSlot * 4, kSplitkSc1);
                }
            }
        if (!splitk_arrive(a.counters + cell, pieces, &ticket)) return;
        auto word = [&](int piece, int at) {
            return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsrc, at * 4, piece * kSlot * 4, kSplitkSc1));
        };
        // a piece's share of each row
        __shared__ float weight[kMaxSplits][kRows];
        for (int i = threadIdx.x; i < pieces * kRows; i += kThreads) {
            const int piece = i / kRows, row = i % kRows;
            if (row < live) {
                share[piece][row] = word(piece, kRows * D + row);
                weight[piece][row] = word(piece, kRows * (D + 1) + row);
            }
        }
        __syncthreads();
        if (int(threadIdx.x) < live) {
            const int row = threadIdx.x;
            float top = kNone, sum = 0.0f;
            for (int p = 0; p < pieces; ++p) top = fmaxf(top, share[p][row]);
            for (int p = 0; p < pieces; ++p) {
                const float w = share[p][row] == kNone ? 0.0f : __builtin_amdgcn_exp2f(share[p][row] - top);
                share[p][row] = w;
                sum = fmaf(weight[p][row], w, sum);
            }
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
            for (int p = 0; p < pieces; ++p) share[p][row] *= inv;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < live * (D / 4); i += kThreads) {
            const int row = i / (D / 4), at = row * D + i % (D / 4) * 4;
            f4 sum = {0, 0, 0, 0};
            for (int p = 0; p < pieces; ++p) {
                const f4 v = __builtin_bit_cast(f4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at * 4, p * kSlot * 4, kSplitkSc1));
                const float w = share[p][row];
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[j] = fmaf(v[j], w, sum[j]);
            }
            *reinterpret_cast<f4*>(out_of(row0 + row) + i % (D / 4) * 4) = sum;
        }
    }
}

// How a call is cut.  Rows enough to fill the card four waves of rows at a time: KW = 1; else the waves of a
// workgroup divide the keys, and workgroups too where there are few tiles.
struct Plan {
    int rt, kw, tiles, splits, chunk_steps;
    int64_t blocks;
};
Plan plan(int64_t seqs, int64_t q_heads, int64_t heads, int64_t max_q, int64_t max_kv) {
    Plan p;
    const int64_t rows = max_q * (q_heads / heads), steps = (max_kv + kStep - 1) / kStep + 1;
    p.rt = rows <= 16 ? 1 : 2;
    const int64_t wide = (rows + 16 * p.rt * kWaves - 1) / (16 * p.rt * kWaves);
    p.kw = rows >= 16 * p.rt * kWaves && seqs * heads * wide >= kTarget ? 1 : kWaves;
    const int64_t tiles = p.kw == 1 ? wide : (rows + 16 * p.rt - 1) / (16 * p.rt);
    const int64_t items = seqs * heads * tiles;
    int64_t splits = 1;
    if (p.kw > 1 && items < kTarget)
        splits = std::max<int64_t>(1, std::min<int64_t>({int64_t(kMaxSplits), kTarget / items, steps / (kMinSteps * kWaves)}));
    p.chunk_steps = int((steps + splits - 1) / splits);
    p.splits = int((steps + p.chunk_steps - 1) / p.chunk_steps);
    p.tiles = int(tiles);
    p.blocks = items * p.splits;
    return p;
}

size_t slot_floats(const Plan& p, int64_t dim) { return size_t(16 * p.rt) * size_t(dim + 2); }

}  // namespace

size_t attn_scratch_bytes(int, int64_t seqs, int64_t q_heads, int64_t heads, int64_t dim, int64_t max_q, int64_t max_kv) {
    const Plan p = plan(seqs, q_heads, heads, max_q, max_kv);
    return size_t(kCounters) * 4 + (p.splits > 1 ? size_t(p.blocks) * slot_floats(p, dim) * 4 : 0);
}

bool attn_fits(int64_t seqs, int64_t q_heads, int64_t heads, int64_t max_q, int64_t max_kv) {
    return plan(seqs, q_heads, heads, max_q, max_kv).blocks < (int64_t(1) << 31);
}

hipError_t launch_attn(const Attn& r, hipStream_t s, const char** name) {
    const Plan p = plan(r.cache.view.seqs, r.q_heads, r.cache.view.heads, r.max_q, r.max_kv);
    *name = p.kw == 1 ? "attn_rows" : p.splits > 1 ? "attn_split" : "attn_keys";
    AttnArgs a;
    a.c = r.cache.view;
    a.q = r.q;
    a.out = r.out;
    a.counters = static_cast<unsigned*>(r.scratch);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(r.scratch) + size_t(kCounters) * 4);
    a.q_stride = r.q_stride;
    a.T = int(r.T);
    a.q_heads = int(r.q_heads);
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
    auto shape = [&](auto bits, auto dim) {
        constexpr int kB = decltype(bits)::value, kD = decltype(dim)::value;
        if (p.kw == 1) p.rt == 1 ? run(attn_kernel<kB, kD, 1, 1>) : run(attn_kernel<kB, kD, 2, 1>);
        else p.rt == 1 ? run(attn_kernel<kB, kD, 1, kWaves>) : run(attn_kernel<kB, kD, 2, kWaves>);
    };
    kv_kinds(r.cache.bits, r.cache.dim, shape);
    return hipGetLastError();
}

}  // namespace mq
