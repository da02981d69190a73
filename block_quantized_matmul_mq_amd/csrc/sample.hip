// mq_sample: a token per row of logits by temperature, top-k, top-p and min-p, from a given random number.
//
//   e_i = exp((l_i - l_max) / T); the tokens in falling order of l (of equal ones the lower index first)
//   kept: the first n = min(top_k, the shortest prefix with mass >= top_p * mass(first top_k), #(e_i >= min_p))
//   the choice: the first kept token, in index order, with  sum of the kept e up to it > u * sum of all kept e
//
// Masses are sums of w_i = rne(2^43 e_i) in 64-bit integers: the order of the sums does not matter, and
// 2^20 tokens fit.  A token with e_i < 2^-44 is never chosen.  The kept set is a key (the logit's bits in
// the order of its value) and a count of tokens that have exactly this key, found by radix selection.
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr double kUnit = 8796093022208.0;   // 2^43
typedef unsigned long long u64;

// Keys in the order of the logits; 0 for a NaN and for -inf, which are never chosen.
__device__ __forceinline__ uint32_t key_of(float l) {
    if (!(l > -__builtin_inff())) return 0;
    const uint32_t u = __builtin_bit_cast(uint32_t, l + 0.0f);   // -0 is 0
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7FFFFFFFu : ~key);
}

struct Row {
    const float* l;
    int V;
    double top, inv;   // the largest logit, 1 / T
};

// e of a logit: 1 for the largest one (also an infinity)
__device__ __forceinline__ double weight(const Row& r, float l) {
    const double x = (double(l) - r.top) * r.inv;
    return double(l) == r.top ? 1.0 : exp(x);
}
__device__ __forceinline__ u64 mass(double e) { return u64(rint(e * kUnit)); }

struct Smem {
    u64 w[kBins];
    uint32_t n[kBins];
    u64 wave_w[kWaves];
    uint32_t wave_n[kWaves];
    uint32_t key, skip, bin;
    u64 above_w, total;
    uint32_t above_n;
    int id;
    double e;
};

// The key at which the prefix ends: by count (the `limit`-th token), or by mass (the first at which the sum
// reaches `goal`).  above_n, above_w: tokens of larger keys; floor: smaller keys do not count.
__device__ void select(const Row& r, Smem& sm, bool by_mass, double goal, uint32_t limit, uint32_t floor_key) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        sm.above_n = 0;
        sm.above_w = 0;
        sm.key = 0;
    }
    const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = shifts[pass], bins = 1 << widths[pass];
        __syncthreads();
        for (int b = tid; b < kBins; b += kThreads) {
            sm.n[b] = 0;
            sm.w[b] = 0;
        }
        __syncthreads();
        const uint32_t prefix = sm.key;
        const int above = shift + widths[pass];
        for (int i = tid; i < r.V; i += kThreads) {
            const float l = r.l[i];
            const uint32_t key = key_of(l);
            if (key == 0 || key < floor_key || (above < 32 && (key >> above) != (prefix >> above))) continue;
            const int b = (key >> shift) & (bins - 1);
            atomicAdd(&sm.n[b], 1u);
            atomicAdd(&sm.w[b], mass(weight(r, l)));
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t n = sm.above_n;
            u64 w = sm.above_w;
            int b = bins - 1, last = -1;
            for (; b >= 0; --b) {
                if (sm.n[b] == 0) continue;
                last = b;
                if (by_mass ? double(w + sm.w[b]) >= goal : n + sm.n[b] >= limit) break;
                n += sm.n[b];
                w += sm.w[b];
            }
            if (b < 0) {   // every token is in: end at the lowest bin that has one
                b = last < 0 ? 0 : last;
                n -= last < 0 ? 0 : sm.n[b];
                w -= last < 0 ? 0 : sm.w[b];
            }
            sm.above_n = n;
            sm.above_w = w;
            sm.key = prefix | uint32_t(b) << shift;
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(kThreads) void sample_kernel(Sample a) {
    __shared__ Smem sm;
    const int m = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Row r = {a.logits + m * a.stride, int(a.V), 0.0, 0.0};
    // the largest logit, and its first index
    u64 best = 0;
    for (int i = tid; i < r.V; i += kThreads) {
        const u64 k = u64(key_of(r.l[i])) << 32 | uint32_t(~i);
        best = k > best ? k : best;
    }
    for (int off = 32; off; off >>= 1) {
        const u64 o = __shfl_xor(best, off, 64);
        best = o > best ? o : best;
    }
    if (lane == 0) sm.wave_w[wave] = best;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) best = sm.wave_w[w] > best ? sm.wave_w[w] : best;
    const uint32_t top_key = uint32_t(best >> 32);
    const float T = a.temperature ? a.temperature[m] : 1.0f;
    if (top_key == 0 || !(T > 0.0f)) {
        if (tid == 0) {
            a.ids[m] = top_key == 0 ? -1 : int(~uint32_t(best));
            if (a.probs) a.probs[m] = top_key == 0 ? 0.0f : 1.0f;
        }
        return;
    }
    r.top = double(logit_of(top_key));
    r.inv = 1.0 / double(T);
    // the kept set: keys above `key`, and the first `ties` tokens that have it
    uint32_t key = 1, ties = 0xFFFFFFFFu;
    const int k = a.top_k ? a.top_k[m] : 0;
    if (k > 0 && k < r.V) {
        select(r, sm, false, 0.0, uint32_t(k), 1);
        key = sm.key;
        ties = uint32_t(k) - sm.above_n;
    }
    const float p = a.top_p ? a.top_p[m] : 1.0f;
    if (p < 1.0f) {
        // the mass of the first top_k
        u64 w = 0;
        for (int i = tid; i < r.V; i += kThreads) {
            const uint32_t ki = key_of(r.l[i]);
            if (ki != 0 && (ties == 0xFFFFFFFFu ? ki >= key : ki > key)) w += mass(weight(r, r.l[i]));
        }
        for (int off = 32; off; off >>= 1) w += __shfl_xor(w, off, 64);
        __syncthreads();
        if (lane == 0) sm.wave_w[wave] = w;
        __syncthreads();
        w = 0;
        for (int i = 0; i < kWaves; ++i) w += sm.wave_w[i];
        if (ties != 0xFFFFFFFFu) w += ties * mass(weight(r, logit_of(key)));
        const double goal = double(p) * double(w);
        select(r, sm, true, goal, 0, key);
        if (sm.key != key || ties == 0xFFFFFFFFu) ties = 0xFFFFFFFFu;
        key = sm.key;
        const double each = double(mass(weight(r, logit_of(key))));
        const double lack = goal - double(sm.above_w);
        uint32_t n = lack > 0.0 && each > 0.0 ? uint32_t(fmin(ceil(lack / each), 4294967040.0)) : lack > 0.0 ? ties : 0;
        if (n == 0 && key == top_key) n = 1;
        ties = n < ties ? n : ties;
    }
    const float mp = a.min_p ? a.min_p[m] : 0.0f;
    const float low = mp < 1.0f ? mp : mp >= 1.0f ? 1.0f : 0.0f;   // (a NaN: none)
    // the kept tokens' masses by wave: a wave's share is one run of whole 64s
    const int share = ((r.V + 63) / 64 + kWaves - 1) / kWaves * 64;
    const int from = wave * share, to = from + share < r.V ? from + share : r.V;
    uint32_t tied = 0;
    for (int i = from + lane; i < to; i += 64) tied += key_of(r.l[i]) == key;
    for (int off = 32; off; off >>= 1) tied += __shfl_xor(tied, off, 64);
    __syncthreads();
    if (lane == 0) sm.wave_n[wave] = tied;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < wave; ++w) before += sm.wave_n[w];
    auto kept = [&](int i, uint32_t& seen, double& e) {   // all lanes call; seen: ties before the 64 tokens
        const float l = i < to ? r.l[i] : 0.0f;
        const uint32_t ki = i < to ? key_of(l) : 0;
        const u64 same = __ballot(ki == key);
        const uint32_t rank = seen + __popcll(same & ((u64(1) << lane) - 1));
        seen += __popcll(same);
        if (ki == 0 || ki < key || (ki == key && rank >= ties)) return u64(0);
        e = weight(r, l);
        return ki != top_key && e < double(low) ? u64(0) : mass(e);
    };
    u64 sum = 0;
    uint32_t seen = before;
    double e = 0.0;
    for (int i = from; i < to; i += 64) sum += kept(i + lane, seen, e);
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) sm.wave_w[wave] = sum;
    __syncthreads();
    u64 total = 0, upto = 0;
    for (int w = 0; w < kWaves; ++w) total += sm.wave_w[w];
    double u = double(a.u[m]);
    u = u > 0.0 ? u : 0.0;
    const u64 goal = u < 1.0 ? u64(floor(u * double(total))) : ~u64(0);
    const u64 need = goal < total - 1 ? goal : total - 1;   // the first token whose sum passes this
    for (int w = 0; w < wave; ++w) upto += sm.wave_w[w];
    if (need < upto || need >= upto + sum) return;
    seen = before;
    for (int i = from; i < to; i += 64) {
        const u64 w = kept(i + lane, seen, e);
        u64 run = w;
        for (int off = 1; off < 64; off <<= 1) {
            const u64 o = __shfl_up(run, off, 64);
            if (lane >= off) run += o;
        }
        if (w != 0 && upto + run > need && upto + run - w <= need) {
            a.ids[m] = i + lane;
            if (a.probs) a.probs[m] = float(e / (double(total) / kUnit));
        }
        upto += __shfl(run, 63, 64);
        if (upto > need) break;
    }
}

}  // namespace

size_t sample_scratch_bytes(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const Sample& r, hipStream_t s, const char** name) {
    *name = "sample";
    hipLaunchKernelGGL(sample_kernel, dim3(unsigned(r.M)), dim3(kThreads), 0, s, r);
    return hipGetLastError();
}

}  // namespace mq
