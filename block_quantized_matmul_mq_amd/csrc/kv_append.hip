// mq_kv_append: the heads' norm, the position rotation and the append of keys and values to the paged
// cache, in one pass over a decoder layer's q, k and v; mq_kv_read: rows of the cache as f32.
//
//   y = x w / sqrt(mean(x^2) + eps)                            (q and k, where a norm is given)
//   (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a),  a = pos inv_freq[j]
//   K, V: blocks of 32, 4 bits: d = f16(m / -8), m the value of largest magnitude with its sign,
//   code = clamp(rne(x / d) + 8, 0, 15); 8 bits: d = f16(amax / 127), code = clamp(rne(x / d), -127, 127) + 128
//
// Norm and rotation are formed in f64 and rounded once to f32: a key's code flips where its last f32 bit
// does, and so the cache is the formula's byte for byte (an f32 form in this order of sums would depend on
// the batch as little, but flip single codes).
//
// A row (a head of a token) to a wave, the values in the lanes of the block that they belong to: a block's maximum and the
// norm's sum are lane reductions, and a wave that takes several rows of a token forms its angles once.  Few tokens: 4 us, a
// launch's latency.  Three prompts, 2980 tokens of 40 + 2 x 8 heads of 128, normed: 46.5 us, 3.2 TB/s (a copy here has 4.7), the vector ALU busy
// for 58 to 63 % of it, mostly with f64; reading the 4-bit cache back as f32 11.5 us.
#include "kv_layout.h"
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

constexpr int kWaves = 4;

struct AppendArgs {
    KvView c;
    const float *q, *k, *v, *q_norm, *k_norm, *inv_freq;
    const int32_t* pos;
    float* q_out;
    int64_t q_stride, k_stride, v_stride, out_stride;
    int q_heads, rot, rope;
    float eps;
};

// cos and sin of a >= 0 or < 0 in f64: a - n pi/2 with pi/2 as two doubles (the fma is exact in the first),
// then both Taylor series on [-pi/4, pi/4] (the first terms left out are below 2^-53).
__device__ __forceinline__ void sincos64(double a, double& s, double& c) {
    const double n = rint(a * 0.63661977236758134308);
    double r = fma(-n, 1.57079632679489655800, a);
    r = fma(-n, 6.12323399573676603587e-17, r);
    const double z = r * r;
    double ps = -1.0 / 1307674368000.0;
    ps = fma(ps, z, 1.0 / 6227020800.0);
    ps = fma(ps, z, -1.0 / 39916800.0);
    ps = fma(ps, z, 1.0 / 362880.0);
    ps = fma(ps, z, -1.0 / 5040.0);
    ps = fma(ps, z, 1.0 / 120.0);
    ps = fma(ps, z, -1.0 / 6.0);
    ps = fma(ps * z, r, r);
    double pc = 1.0 / 20922789888000.0;
    pc = fma(pc, z, -1.0 / 87178291200.0);
    pc = fma(pc, z, 1.0 / 479001600.0);
    pc = fma(pc, z, -1.0 / 3628800.0);
    pc = fma(pc, z, 1.0 / 40320.0);
    pc = fma(pc, z, -1.0 / 720.0);
    pc = fma(pc, z, 1.0 / 24.0);
    pc = fma(pc, z, -0.5);
    pc = fma(pc, z, 1.0);
    const int64_t k = int64_t(n);
    s = k & 1 ? pc : ps;
    c = k & 1 ? ps : pc;
    if (k & 2) s = -s;
    if ((k + 1) & 2) c = -c;
}

// 1 / sqrt(v) of a normal v > 0: the instruction's 2^-26 or so and two Newton steps, each of which squares that.
__device__ __forceinline__ double inverse_sqrt(double v) {
    double y = __builtin_amdgcn_rsq(v);
#pragma unroll
    for (int i = 0; i < 2; ++i) y = fma(fma(-v * y, y, 1.0), 0.5 * y, y);
    return y;
}

// Lanes l and l ^ 1, 2 and the other quad of eight, the other eight of sixteen: DPP moves; 16 and 32 apart: swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(v), CTRL, 0xF, 0xF, false));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kQuads = 0x141, kEights = 0x140;
template <int STEP>
__device__ __forceinline__ void swapped(uint32_t v, uint32_t& a, uint32_t& b) {
    const auto x = STEP == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false) : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = x[0];
    b = x[1];
}
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return v + __builtin_bit_cast(double, uint64_t(dpp<CTRL>(uint32_t(u >> 32))) << 32 | dpp<CTRL>(uint32_t(u)));
}
template <int STEP>
__device__ __forceinline__ double add_swapped(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t la, lb, ha, hb;
    swapped<STEP>(uint32_t(u), la, lb);
    swapped<STEP>(uint32_t(u >> 32), ha, hb);
    return __builtin_bit_cast(double, uint64_t(ha) << 32 | la) + __builtin_bit_cast(double, uint64_t(hb) << 32 | lb);
}
__device__ __forceinline__ double wave_sum64(double v) {
    v = add_dpp<kEights>(add_dpp<kQuads>(add_dpp<kXor2>(add_dpp<kXor1>(v))));
    return add_swapped<32>(add_swapped<16>(v));
}
template <int CTRL>
__device__ __forceinline__ float max_dpp(float v) {
    return fmaxf(v, __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v))));
}
// over aligned groups of 32 lanes
__device__ __forceinline__ float max32(float v) {
    v = max_dpp<kEights>(max_dpp<kQuads>(max_dpp<kXor2>(max_dpp<kXor1>(v))));
    uint32_t a, b;
    swapped<16>(__builtin_bit_cast(uint32_t, v), a, b);
    return fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
}

// One block per 32 lanes: the scale (f16 bits) and this lane's code of x.
template <int BITS>
__device__ __forceinline__ int quantize(float x, uint32_t& d_bits) {
    const int lane = threadIdx.x & 63;
    const float big = max32(fabsf(x));
    const bool bad = !(fabsf(x) <= 3.4028235e38f);
    const unsigned long long half = 0xFFFFFFFFull << (lane & 32);
    const bool any_bad = (__ballot(bad) & half) != 0;
    _Float16 d;
    if constexpr (BITS == 4) {
        // the sign of the first value of largest magnitude
        const unsigned long long who = __ballot(fabsf(x) == big) & half, negative = __ballot(x < 0.0f);
        const bool minus = who != 0 && (negative >> (__ffsll(who) - 1) & 1);
        d = static_cast<_Float16>((minus ? -big : big) / -8.0f);
    } else {
        d = static_cast<_Float16>(big / 127.0f);
    }
    const float df = static_cast<float>(d);
    // a block with an infinity or a NaN, or past f16's range, reads as NaN
    if (any_bad || !(fabsf(df) <= 65504.0f)) {
        d_bits = 0x7E00u;
        return BITS == 4 ? 8 : 128;
    }
    if (df == 0.0f) {
        d_bits = 0;
        return BITS == 4 ? 8 : 128;
    }
    d_bits = __builtin_bit_cast(uint16_t, d);
    const float r = rintf(x / df);
    if constexpr (BITS == 4) return int(fminf(fmaxf(r + 8.0f, 0.0f), 15.0f));
    return int(fminf(fmaxf(r, -127.0f), 127.0f)) + 128;
}

// A wave per row (a head of a token's q, k or v), some rows one after another, the next one's values in flight; lane l holds
// dimensions l + 64 i.  One decoded token of the 7B layer (28 + 8 rows): a row a wave over nine workgroups.
template <int BITS, int D>
__global__ __launch_bounds__(64 * kWaves) void kv_append_kernel(AppendArgs a) {
    using L = KvLayout<BITS, D>;
    constexpr int R = D / 64;
    __shared__ double row[kWaves][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x;
    const int q_rows = a.q ? a.q_heads : 0, kv = a.c.heads, rows = q_rows + 2 * kv, step = kWaves * gridDim.y;
    auto load = [&](int r, float (&x)[R]) {
        const bool is_q = r < q_rows, is_v = r >= q_rows + kv;
        const float* from = is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride;
        from += int64_t(is_q ? r : is_v ? r - q_rows - kv : r - q_rows) * D;
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = from[lane + 64 * i];
    };
    const int first = blockIdx.y * kWaves + wave;
    if (first >= rows) return;
    float next[R];
    load(first, next);
    const KvToken tok = kv_token(a.c, t);
    if (tok.seq < 0) return;
    const int page = kv_page(a.c, tok.seq, tok.pos);
    const int slot = tok.pos & (a.c.page_tokens - 1);
    double sn[R], cs[R];
    int partner[R];
    if (a.rope) {
        const double pos = a.pos ? double(a.pos[t]) : double(tok.pos);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int d = lane + 64 * i, h = a.rot / 2;
            sn[i] = 0.0;
            cs[i] = 1.0;
            partner[i] = d;
            if (d < a.rot) {
                const bool lower = a.rope == 1 ? d < h : (d & 1) == 0;
                partner[i] = a.rope == 1 ? (lower ? d + h : d - h) : d ^ 1;
                sincos64(pos * double(a.inv_freq[a.rope == 1 ? (lower ? d : d - h) : d >> 1]), sn[i], cs[i]);
                if (lower) sn[i] = -sn[i];
            }
        }
    }
    float wq[R], wk[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        wq[i] = a.q_norm ? a.q_norm[lane + 64 * i] : 1.0f;
        wk[i] = a.k_norm ? a.k_norm[lane + 64 * i] : 1.0f;
    }
    // pairs of halves that lie in one lane need no exchange
    const bool own = R > 1 && a.rope == 1 && a.rot == D;
    for (int r = first; r < rows; r += step) {
        const bool is_q = r < q_rows, is_v = r >= q_rows + kv;
        const int h = is_q ? r : is_v ? r - q_rows - kv : r - q_rows;
        float x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = next[i];
        if (r + step < rows) load(r + step, next);
        if (!is_q && page < 0) continue;
        const float* w = is_q ? a.q_norm : a.k_norm;
        if (!is_v && (w || a.rope)) {
            double y[R];
#pragma unroll
            for (int i = 0; i < R; ++i) y[i] = x[i];
            if (w) {
                double s = 0.0;
#pragma unroll
                for (int i = 0; i < R; ++i) s = fma(y[i], y[i], s);
                s = fma(wave_sum64(s), 1.0 / D, double(a.eps));
                s = s >= 0x1p-1000 && s <= 0x1p1000 ? inverse_sqrt(s) : 1.0 / sqrt(s);
#pragma unroll
                for (int i = 0; i < R; ++i) y[i] = y[i] * s * double(is_q ? wq[i] : wk[i]);
            }
            if (own) {
                double z[R];
#pragma unroll
                for (int i = 0; i < R; ++i) z[i] = fma(y[i], cs[i], y[(i + R / 2) % R] * sn[i]);
#pragma unroll
                for (int i = 0; i < R; ++i) y[i] = z[i];
            } else if (a.rope) {
#pragma unroll
                for (int i = 0; i < R; ++i) row[wave][lane + 64 * i] = y[i];
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < R; ++i)
                    if (lane + 64 * i < a.rot) y[i] = fma(y[i], cs[i], row[wave][partner[i]] * sn[i]);
                __builtin_amdgcn_wave_barrier();
            }
#pragma unroll
            for (int i = 0; i < R; ++i) x[i] = float(y[i]);
        }
        if (is_q) {
#pragma unroll
            for (int i = 0; i < R; ++i) a.q_out[t * a.out_stride + int64_t(h) * D + lane + 64 * i] = x[i];
            continue;
        }
        uint8_t* chunk = a.c.data + (int64_t(page) * kv + h) * a.c.chunk;
        const int64_t section = int64_t(a.c.page_tokens) * L::kRow;
        uint8_t* codes = chunk + (is_v ? section : 0);
        uint16_t* scales = reinterpret_cast<uint16_t*>(chunk + 2 * section) +
                           (int64_t(is_v) * a.c.page_tokens + slot) * L::kBlocks;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int dim = lane + 64 * i;
            uint32_t d;
            const uint32_t code = uint32_t(quantize<BITS>(x[i], d));
            if ((lane & 31) == 0) scales[dim / 32] = uint16_t(d);
            if (!is_v) {    // 8 or 4 lanes fill a dword
                constexpr int kPer = 32 / BITS;
                uint32_t v = code << (BITS * (lane % kPer));
                v |= dpp<kXor1>(v);
                v |= dpp<kXor2>(v);
                if constexpr (kPer == 8) v |= dpp<kQuads>(v);
                if (lane % kPer == 0) *reinterpret_cast<uint32_t*>(codes + L::k_byte(slot, dim)) = v;
            } else {        // lanes 16 apart fill two bytes
                constexpr int kPer = 16 / BITS;
                uint32_t p, q;
                swapped<16>(code << (BITS * (lane / 16 % kPer)), p, q);
                uint32_t v = p | q;
                if constexpr (kPer == 4) {
                    swapped<32>(v, p, q);
                    v = p | q;
                }
                if (lane / 16 % kPer == 0) *reinterpret_cast<uint16_t*>(codes + L::v_byte(slot, dim)) = uint16_t(v);
            }
        }
    }
}

// A wave per token and head's row (k or v); lane l gives dimensions l + 64 i.
template <int BITS, int D>
__global__ __launch_bounds__(64 * kWaves) void kv_read_kernel(KvView c, float* k, float* v) {
    using L = KvLayout<BITS, D>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x;
    const KvToken tok = kv_token(c, t);
    if (tok.seq < 0) return;
    const int page = kv_page(c, tok.seq, tok.pos);
    const int slot = tok.pos & (c.page_tokens - 1);
    const int64_t section = int64_t(c.page_tokens) * L::kRow;
    for (int r = blockIdx.y * kWaves + wave; r < 2 * c.heads; r += kWaves * gridDim.y) {
        const bool is_v = r >= c.heads;
        const int h = is_v ? r - c.heads : r;
        float* out = is_v ? v : k;
        if (!out) continue;
        out += (int64_t(t) * c.heads + h) * D;
        const uint8_t* chunk = c.data + (int64_t(max(page, 0)) * c.heads + h) * c.chunk;
        const uint16_t* scales = reinterpret_cast<const uint16_t*>(chunk + 2 * section) +
                                 (int64_t(is_v) * c.page_tokens + slot) * L::kBlocks;
        float x[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int dim = lane + 64 * i;
            int code = chunk[is_v ? section + L::v_byte(slot, dim) : L::k_byte(slot, dim)];
            if constexpr (BITS == 4) code = (code >> (4 * (is_v ? L::v_nibble(dim) : L::k_nibble(dim)))) & 15;
            x[i] = float(code - L::kOffset) * half_bits_to_float(scales[dim / 32]);
        }
#pragma unroll
        for (int i = 0; i < D / 64; ++i) out[lane + 64 * i] = page < 0 ? 0.0f : x[i];
    }
}

// Workgroups that share a token's rows: enough for kWavesWanted waves where there are few tokens, a row a wave at least.
constexpr int64_t kWavesWanted = 8192;
unsigned row_groups(int64_t T, int64_t rows) {
    const int64_t most = (rows + kWaves - 1) / kWaves, want = kWavesWanted / (T * kWaves);
    return unsigned(want < 1 ? 1 : want > most ? most : want);
}

}  // namespace

hipError_t launch_kv_append(const KvAppend& r, hipStream_t s, const char** name) {
    *name = "kv_append";
    const AppendArgs a = {r.cache.view, r.q, r.k, r.v, r.q_norm, r.k_norm, r.inv_freq, r.pos, r.q_out, r.q_stride,
                          r.k_stride, r.v_stride, r.out_stride, int(r.q_heads), int(r.rot), r.rope, r.eps};
    const unsigned groups = row_groups(r.T, (r.q ? r.q_heads : 0) + 2 * r.cache.view.heads);
    kv_kinds(r.cache.bits, r.cache.dim, [&](auto bits, auto dim) {
        hipLaunchKernelGGL((kv_append_kernel<decltype(bits)::value, decltype(dim)::value>), dim3(unsigned(r.T), groups),
                           dim3(64 * kWaves), 0, s, a);
    });
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& cache, int64_t T, float* k, float* v, hipStream_t s, const char** name) {
    *name = "kv_read";
    const unsigned groups = row_groups(T, 2 * cache.view.heads);
    kv_kinds(cache.bits, cache.dim, [&](auto bits, auto dim) {
        hipLaunchKernelGGL((kv_read_kernel<decltype(bits)::value, decltype(dim)::value>), dim3(unsigned(T), groups),
                           dim3(64 * kWaves), 0, s, cache.view, k, v);
    });
    return hipGetLastError();
}

}  // namespace mq
