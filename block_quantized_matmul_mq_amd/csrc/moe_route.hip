// mq_moe_route: the router of a mixture of experts.  logit[m][e] = sum_k X[m][k] Wr[e][k],
// p = softmax over e (or the sigmoid) of the logits, the k largest of p + bias (of the logits when
// there is no bias) per token, and their weights.
//
// The logits are summed in f64: a choice next to a border (two logits within a few f32
// roundings of each other) then falls the same way whatever the order of the sums, and the
// products cost little here: the router's weights are 4 E K bytes, and f64 matrix instructions
// run at the f64 vector rate without the lane reductions (v_mfma_f64_16x16x4: lane l supplies
// row l % 16 and k = l / 16 of both operands; a lane loads four consecutive k as one float4 and
// feeds element j to instruction j, which only permutes the sum).
//
// Split.  A workgroup owns 16 tokens x 32 experts x one of S ranges of K, its 16 waves parts of
// that range, summed in LDS in wave order.  Few tokens leave few such tiles, so K is cut until
// about 256 workgroups run (latency bound: one decoded token reads E K floats that one CU
// could not fetch in time).  Each workgroup stores its partial logits to scratch and counts
// itself in on its token tile's counter (mmq_splitk.h's exchange); the last one adds the
// ranges in order and selects: a wave per token, E / 64 logits per lane, k rounds of a
// maximum over the wave on 64-bit keys that order like the f64 values (ties: lowest index).
//
// One token, K = 2048, E = 64: 7.9 us, all of it latency (0.5 MB); 512 tokens, K = 4096, E = 128: 22 us, of which
// the f64 matrix products are about 7.
#include <algorithm>
#include <type_traits>

#include "mmq_splitk.h"
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

typedef double v4d __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kTileM = 16, kTileE = 32;
constexpr int kStep = 16;                     // K values per wave step (K % 32 == 0)
constexpr int kTargetWorkgroups = 256;
// Steps of a wave at least: one where there is one token tile, else two, for fewer ranges that the last
// workgroup has to add (K = 4096, E = 128: one token 8.3 us with one step, 9.3 with two; 64 tokens 19.2 and 17.4).
constexpr int kMinStepsFew = 1, kMinSteps = 2;
constexpr int kCounters = 65536;              // token tiles: MQ_MAX_M / 16
constexpr uint64_t kTaken = 0;

struct RouteArgs {
    const float *X, *Wr, *bias;
    int32_t* ids;
    float* wts;
    double* partial;        // [token tile][range][16][E]
    unsigned* counters;     // [token tile]
    int M, K, E, topk, score, norm, etiles, ranges;
    float scale;
};

// f64 -> unsigned key in the same order; NaN below everything (kTaken, 0, is below that).
__device__ __forceinline__ uint64_t key_of(double v) {
    if (!(v == v)) return 1;
    v += 0.0;   // -0 orders as 0
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    const uint32_t lo = uint32_t(__builtin_amdgcn_mov_dpp(int(uint32_t(v)), CTRL, 0xF, 0xF, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_mov_dpp(int(uint32_t(v >> 32)), CTRL, 0xF, 0xF, false));
    return (uint64_t(hi) << 32) | lo;
}
// The values of lanes l ^ 16 (or l ^ 32) and l, in some order that is the same for both.
template <int STEP>
__device__ __forceinline__ void swap_u64(uint64_t v, uint64_t& a, uint64_t& b) {
    const uint32_t l = uint32_t(v), h = uint32_t(v >> 32);
    if constexpr (STEP == 16) {
        const auto x = __builtin_amdgcn_permlane16_swap(l, l, false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(h, h, false, false);
        a = (uint64_t(y[0]) << 32) | x[0];
        b = (uint64_t(y[1]) << 32) | x[1];
    } else {
        const auto x = __builtin_amdgcn_permlane32_swap(l, l, false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(h, h, false, false);
        a = (uint64_t(y[0]) << 32) | x[0];
        b = (uint64_t(y[1]) << 32) | x[1];
    }
}
// op over all lanes, in registers (no LDS trips)
template <class T, class Op>
__device__ __forceinline__ T wave_all(T v, const Op& op) {
    auto bits = [](T x) { return __builtin_bit_cast(uint64_t, x); };
    auto value = [](uint64_t x) { return __builtin_bit_cast(T, x); };
    v = op(v, value(dpp_u64<0xB1>(bits(v))));    // lane ^ 1
    v = op(v, value(dpp_u64<0x4E>(bits(v))));    // lane ^ 2
    v = op(v, value(dpp_u64<0x141>(bits(v))));   // the other quad of eight
    v = op(v, value(dpp_u64<0x140>(bits(v))));   // the other eight of sixteen (row mirror)
    uint64_t a, b;
    swap_u64<16>(bits(v), a, b);
    v = op(value(a), value(b));
    swap_u64<32>(bits(v), a, b);
    return op(value(a), value(b));
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    return wave_all(v, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ double lane_f64(double v, int lane) {   // lane: uniform
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u)), lane));
    const uint32_t hi = uint32_t(__builtin_amdgcn_readlane(int(uint32_t(u >> 32)), lane));
    return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}

// One token's choices: lane l holds the logits of experts l, l + 64, ...
template <int PER>
__device__ __forceinline__ void select(const RouteArgs& a, int m, const double (&z)[PER], int lane) {
    double p[PER];
    uint64_t key[PER];
    const bool softmax = a.score == 0;
    double top = -__builtin_inf();
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (64 * i + lane < a.E) {
            top = fmax(top, z[i]);
            nan |= !(z[i] == z[i]);
        }
    top = wave_all(top, [](double x, double y) { return fmax(x, y); });
    // The softmax's sum holds every expert's exp: a NaN logit makes all of them NaN, also where only the chosen
    // ones' are summed below.
    if (__ballot(nan) != 0) top = __builtin_nan("");
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        p[i] = 0.0;
        key[i] = kTaken;
        if (e < a.E) {
            p[i] = softmax ? exp(z[i] - top) : 1.0 / (1.0 + exp(-z[i]));
            sum += p[i];
        }
        if constexpr (PER > 4) __builtin_amdgcn_sched_barrier(0);   // one exp at a time (registers)
    }
    if (softmax && (a.bias || !a.norm)) {
        sum = wave_all(sum, [](double x, double y) { return x + y; });
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            p[i] /= sum;
            if constexpr (PER > 4) __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        if (e < a.E) key[i] = key_of(a.bias ? p[i] + double(a.bias[e]) : z[i]);
    }
    double chosen = 0.0, mine = 0.0;   // the sum of the chosen p; lane j: choice j's p
    int my_id = 0;
    for (int j = 0; j < a.topk; ++j) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint64_t all = wave_max(best);
        // the lowest index among the lanes that hold the maximum
        unsigned long long who = __ballot(best == all);
        int e = 64 * at + lane;
        if (who & (who - 1)) {
            int low = best == all ? e : 0x7FFFFFFF;
            for (int off = 1; off < 64; off <<= 1) low = min(low, __shfl_xor(low, off, 64));
            who = __ballot(best == all && e == low);
        }
        const int src = __builtin_amdgcn_readfirstlane(__ffsll(who) - 1);
        double pv = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == at) {
                pv = p[i];
                if (lane == src) key[i] = kTaken;
            }
        e = __builtin_amdgcn_readlane(e, src);
        pv = lane_f64(pv, src);
        chosen += pv;
        if (lane == j) {
            mine = pv;
            my_id = e;
        }
    }
    if (lane < a.topk) {
        const double w = a.norm ? mine / chosen : mine;
        a.ids[int64_t(m) * a.topk + lane] = my_id;
        a.wts[int64_t(m) * a.topk + lane] = float(w * double(a.scale));
    }
}

// PER: logits a lane holds when the last workgroup selects (E <= 64 PER).
template <int PER>
__global__ __launch_bounds__(kThreads) void moe_route_kernel(RouteArgs a) {
    __shared__ double red[kWaves][kTileM * kTileE];   // 64 KiB: the waves' partial tiles
    __shared__ unsigned ticket;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int per_tile = a.etiles * a.ranges;
    const int mt = blockIdx.x / per_tile, rest = blockIdx.x - mt * per_tile;
    const int et = rest % a.etiles, range = rest / a.etiles;
    const int m0 = mt * kTileM, e0 = et * kTileE;
    const int r = lane & 15, q = lane >> 4;
    // K steps of this range, then of this wave
    const int steps = a.K / kStep;
    const int rb = int(int64_t(range) * steps / a.ranges), re = int(int64_t(range + 1) * steps / a.ranges);
    const int sb = rb + (re - rb) * wave / kWaves, se = rb + (re - rb) * (wave + 1) / kWaves;
    // rows past the last re-read it (their results are not used)
    const float* x = a.X + int64_t(min(m0 + r, a.M - 1)) * a.K + 4 * q;
    const float* w0 = a.Wr + int64_t(min(e0 + r, a.E - 1)) * a.K + 4 * q;
    const float* w1 = a.Wr + int64_t(min(e0 + 16 + r, a.E - 1)) * a.K + 4 * q;
    v4d c0 = {0, 0, 0, 0}, c1 = c0;
#pragma unroll 4
    for (int s = sb; s < se; ++s) {
        const float4 xv = *reinterpret_cast<const float4*>(x + kStep * s);
        const float4 u = *reinterpret_cast<const float4*>(w0 + kStep * s);
        const float4 v = *reinterpret_cast<const float4*>(w1 + kStep * s);
        const float xs[4] = {xv.x, xv.y, xv.z, xv.w}, us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c0 = __builtin_amdgcn_mfma_f64_16x16x4f64(double(xs[j]), double(us[j]), c0, 0, 0, 0);
            c1 = __builtin_amdgcn_mfma_f64_16x16x4f64(double(xs[j]), double(vs[j]), c1, 0, 0, 0);
        }
    }
    // accumulator element i of lane l: token 4 i + l / 16, expert l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        red[wave][(4 * i + q) * kTileE + r] = c0[i];
        red[wave][(4 * i + q) * kTileE + 16 + r] = c1[i];
    }
    __syncthreads();
    const int t = tid / kTileE, e = tid % kTileE;   // the first 512 threads: one element each
    double z = 0.0;
    if (tid < kTileM * kTileE)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) z += red[w][tid];
    double* slots = a.partial + int64_t(mt) * a.ranges * kTileM * a.E;
    const bool ok = t < kTileM && m0 + t < a.M && e0 + e < a.E;
    if (ok)   // written through to the device-coherent level (mmq_splitk.h)
        __hip_atomic_store(slots + (int64_t(range) * kTileM + t) * a.E + e0 + e, z, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    if (!splitk_arrive(a.counters + mt, a.etiles * a.ranges, &ticket)) return;
    // The last workgroup of this token tile: the logits summed over the ranges in order (16 or 4 loads in
    // flight: each is a trip to the device-coherent level), then one token per wave selected from LDS.
    double* logits = &red[0][0];   // [token][E]
    static_assert(sizeof(red) >= sizeof(double) * kWaves * kMoeMaxExperts, "the logits of the tile");
    static_assert(kWaves == kTileM, "a wave per token");
    const int count = min(kTileM, a.M - m0) * a.E;
    for (int i = tid; i < count; i += kThreads) {
        const double* from = slots + i;   // (tokens of a range are E apart, as here)
        double sum = 0.0;
        int g = 0;
        auto batch = [&](auto n_c) {
            constexpr int kN = decltype(n_c)::value;
            for (; g + kN <= a.ranges; g += kN) {
                double v[kN];
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    v[j] = __hip_atomic_load(from + int64_t(g + j) * kTileM * a.E, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int j = 0; j < kN; ++j) sum += v[j];
            }
        };
        batch(std::integral_constant<int, 16>{});
        batch(std::integral_constant<int, 4>{});
        batch(std::integral_constant<int, 1>{});
        logits[i] = sum;
    }
    __syncthreads();
    if (m0 + wave < a.M) {
        double mine[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) mine[i] = logits[wave * a.E + min(64 * i + lane, a.E - 1)];
        select<PER>(a, m0 + wave, mine, lane);
    }
}

template __global__ void moe_route_kernel<1>(RouteArgs);
template __global__ void moe_route_kernel<2>(RouteArgs);
template __global__ void moe_route_kernel<4>(RouteArgs);
template __global__ void moe_route_kernel<8>(RouteArgs);

// Ranges of K: about kTargetWorkgroups workgroups in all.
int route_ranges(int64_t M, int64_t K, int64_t E) {
    const int64_t tiles = ((M + kTileM - 1) / kTileM) * ((E + kTileE - 1) / kTileE);
    return int(std::max<int64_t>(1, std::min<int64_t>(kTargetWorkgroups / tiles, K / (kStep * kWaves * (M <= kTileM ? kMinStepsFew : kMinSteps)))));
}

}  // namespace

size_t moe_route_scratch_bytes(int64_t M, int64_t K, int64_t E) {
    const int64_t mtiles = (M + kTileM - 1) / kTileM;
    return size_t(kCounters) * 4 + size_t(mtiles) * route_ranges(M, K, E) * kTileM * size_t(E) * 8;
}

hipError_t launch_moe_route(const MoeRoute& r, hipStream_t s, const char** name) {
    *name = "moe_route";
    RouteArgs a;
    a.X = r.X;
    a.Wr = r.Wr;
    a.bias = r.bias;
    a.ids = r.ids;
    a.wts = r.wts;
    a.counters = static_cast<unsigned*>(r.scratch);
    a.partial = reinterpret_cast<double*>(static_cast<uint8_t*>(r.scratch) + size_t(kCounters) * 4);
    a.M = int(r.M);
    a.K = int(r.K);
    a.E = int(r.E);
    a.topk = int(r.topk);
    a.score = r.score;
    a.norm = r.norm;
    a.scale = r.scale;
    a.etiles = int((r.E + kTileE - 1) / kTileE);
    a.ranges = route_ranges(r.M, r.K, r.E);
    const dim3 grid(unsigned((r.M + kTileM - 1) / kTileM) * unsigned(a.etiles * a.ranges));
    if (r.E <= 64) hipLaunchKernelGGL(moe_route_kernel<1>, grid, dim3(kThreads), 0, s, a);
    else if (r.E <= 128) hipLaunchKernelGGL(moe_route_kernel<2>, grid, dim3(kThreads), 0, s, a);
    else if (r.E <= 256) hipLaunchKernelGGL(moe_route_kernel<4>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(moe_route_kernel<kMoeMaxExperts / 64>, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace mq
