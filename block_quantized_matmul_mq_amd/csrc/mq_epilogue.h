// Activations, and the epilogue that mq_gemv_ep and mq_gemm_ep apply where a kernel stores its
// result:  y[m][n] = act(acc + bias[n]) * mul[m][n] + residual[m][n]   (absent terms are left out).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mq_device.h"

namespace mq {

constexpr int kActNone = 0;
constexpr int kActSilu = 1;
constexpr int kActGeluTanh = 2;
constexpr int kActGeluErf = 3;
constexpr int kActRelu = 4;
constexpr int kActs = 5;

// 1 / (1 + e^-u).  e^-u as 2^t by the exp2 instruction, t = -u log2(e) rounded to f32, times 1 + r ln 2
// for what the rounding of t left out (r: an fma's exact remainder and log2(e)'s own low part), so
// the relative error stays at a few roundings for large |u| too; then one reciprocal
// instruction, which gives 0 for a quotient below 2^-126 (u < -87.3).  (512 x 18944 x 3584 Q4_K with silu and mul, in a
// captured graph, three weight matrices in turn: 163 us with expf and an IEEE division, 160 with this; 143 is mq_gemm.)  e^-u overflows to infinity (1 / inf = 0; its r
// may be NaN, as that of e^-u = 0) and keeps a NaN.
__device__ __forceinline__ float logistic(float u) {
    constexpr float kLog2e = 1.44269502162933349609375f;        // f32(log2 e)
    constexpr float kLog2eLow = 1.92596299112661746887e-8f;     // log2 e - f32(log2 e)
    constexpr float kLn2 = 0.693147182464599609375f;
    const float t = -u * kLog2e;
    const float r = fmaf(-u, kLog2eLow, fmaf(-u, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_amdgcn_rcpf(1.0f + (e > 0.0f && e < __builtin_inff() ? fmaf(e, r * kLn2, e) : e));
}

// (act is uniform: one branch.  Both gelus in the forms that lose nothing to cancellation for
// negative v: 1 + tanh(u) = 2 / (1 + e^-2u), 1 + erf(t) = erfc(-t).)
__device__ __forceinline__ float activate(float v, int act) {
    switch (act) {
        case kActSilu: return v * logistic(v);
        case kActGeluTanh: return v * logistic(1.5957691216057308f * fmaf(0.044715f * v, v * v, v));
        case kActGeluErf: return 0.5f * v * erfcf(-0.70710678118654752f * v);
        case kActRelu: return v <= 0.0f ? 0.0f : v;   // (the maximum instruction would turn a NaN into 0)
        default: return v;
    }
}

// The products without an epilogue.
struct NoEpilogue {
    static constexpr bool kIs = false;
    __device__ __forceinline__ float operator()(float acc, int64_t, int) const { return acc; }
};

// at: m N + n.  mul and residual may be the output itself: an element is read by the thread
// that then writes it.
struct Epilogue {
    static constexpr bool kIs = true;
    const float* bias;
    const float* mul;
    const float* residual;
    int act;
    __device__ __forceinline__ float operator()(float acc, int64_t at, int n) const {
        float v = bias ? acc + bias[n] : acc;
        v = activate(v, act);
        if (mul) v *= mul[at];
        if (residual) v += residual[at];
        return v;
    }
    // The same for C elements of one column n, at(v) the (valid) place of element v: each term's
    // loads are issued together and before the activations, instead of one round trip per element
    // (512 x 18944 x 3584 Q4_K with silu and mul, measured as logistic above: 215 -> 160 us).
    template <int C, class At>
    __device__ __forceinline__ void column(float (&y)[C], int n, const At& at) const {
        float f[C], r[C];
        float b = 0.f;
        if (bias) b = bias[n];
        if (mul)
#pragma unroll
            for (int v = 0; v < C; ++v) f[v] = mul[at(v)];
        if (residual)
#pragma unroll
            for (int v = 0; v < C; ++v) r[v] = residual[at(v)];
        if (bias)
#pragma unroll
            for (int v = 0; v < C; ++v) y[v] += b;
        // (one branch for the column: with the choice inside the loop the elements run one by one)
        auto all = [&](auto act_c) {
#pragma unroll
            for (int v = 0; v < C; ++v) y[v] = activate(y[v], decltype(act_c)::value);
        };
        if (act == kActSilu) all(std::integral_constant<int, kActSilu>{});
        else if (act == kActGeluTanh) all(std::integral_constant<int, kActGeluTanh>{});
        else if (act == kActGeluErf) all(std::integral_constant<int, kActGeluErf>{});
        else if (act == kActRelu) all(std::integral_constant<int, kActRelu>{});
        if (mul)
#pragma unroll
            for (int v = 0; v < C; ++v) y[v] *= f[v];
        if (residual)
#pragma unroll
            for (int v = 0; v < C; ++v) y[v] += r[v];
    }
};

// The output pointer of a product kernel.  Its epilogue's mul and residual may be the same memory, so only the
// products without one promise the compiler that nothing else reads it.
template <class EP> struct Output { using T = float* __restrict__; };
template <> struct Output<Epilogue> { using T = float*; };

// The epilogue argument of a kernel launched through an argument array (ep null: NoEpilogue's,
// one byte that nothing reads).
inline void* epilogue_arg(const Epilogue* ep) {
    static NoEpilogue none;
    return ep ? const_cast<void*>(static_cast<const void*>(ep)) : static_cast<void*>(&none);
}

// The sum of four activations of a block staged as integers, x = 2^-k rint(2^k x) with |2^k x| <= 2^21: of
// the staged x in the kernels with an epilogue (exact), of x itself in those without, whose results are
// fixed.  A code's offset and a minimum then multiply the same x that the codes meet, so that staging's error of
// x carries through the weight and not through the code (Q4_0, 9872 x 5408: 9.8e-7 -> 5.1e-7 relative).  A value
// that is not finite, whose digits mean nothing, makes the sum a NaN, and so every output.
template <class EP>
__device__ __forceinline__ float staged_sum(const float4 v, int k) {
    if constexpr (!EP::kIs) return (v.x + v.y) + (v.z + v.w);
    constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to whole numbers
    auto rounded = [&](float x) { return (ldexpf(x, k) + kRound) - kRound; };
    return not_finite(v, ldexpf((rounded(v.x) + rounded(v.y)) + (rounded(v.z) + rounded(v.w)), -k));
}

// An f32 (its bits) as three bf16 pieces of 8 bits each, high + mid + low exactly; each piece
// twice in a dword (an MFMA operand meets it with both halves of a hi | lo pair).
struct Bf16x3 {
    uint32_t hh, mm, ll;
};
__device__ __forceinline__ Bf16x3 bf16_split3(uint32_t bits) {
    const uint32_t h = bits & 0xFFFF0000u;
    const float r = __uint_as_float(bits) - __uint_as_float(h);
    const uint32_t m = __float_as_uint(r) & 0xFFFF0000u;
    const uint32_t l = __float_as_uint(r - __uint_as_float(m));
    return Bf16x3{h | (h >> 16), m | (m >> 16), (l & 0xFFFF0000u) | (l >> 16)};
}

}  // namespace mq
