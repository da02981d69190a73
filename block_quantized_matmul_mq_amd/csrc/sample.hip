// mq_sample: a token per row of logits by temperature, top-k, top-p and min-p, from a given random number.
//
//   e_i = exp((l_i - l_max) / T); the tokens in falling order of l (of equal ones the lower index first)
//   kept: the first n = min(top_k, the shortest prefix with mass >= top_p * mass(first top_k), #(e_i >= min_p))
//   the choice: the first kept token, in index order, with  sum of the kept e up to it > u * sum of all kept e
//
// Masses are sums of w_i = rne(2^43 e_i) in 64-bit integers: the order of the sums does not matter, and
// 2^20 tokens fit.  A token with e_i < 2^-44 is never chosen; such tokens (x_i = (l_max - l_i) / T > 44 ln 2) are left
// out everywhere.  e is formed in f64: a draw next to a border has to fall the same way whatever divides the work.
//
// No sort of the row.  A token is ranked by the 64-bit number (bits of l in the order of its value, ~index), so the
// kept prefix is "numbers from `cut` on".  Three passes over the logits:
//   1  the largest number
//   2  counts and masses by 1024 bins of x (each 0.03 wide: a bin's weights differ by 3 %); from these the bins in
//      which the cuts of top-k and top-p lie
//   3  the tokens of these bins, a few hundred, collected; and the masses of 2048-token blocks of the tokens that are in whatever
//      the cuts are.  Then, once a row: the collected tokens sorted, both cuts, the kept ones' masses added to their
//      blocks, the block that the random number falls in, and the token in it.
// A row of more than two blocks is divided over workgroups and the passes over launches (the last workgroup of a row does a
// pass's single part, mmq_splitk.h's exchange); a shorter one is a workgroup's, which makes all passes by itself.
// Measured: one row of 152064 25 us (launches of 3.6, 11.3 and 11.3: latency of their dependent rounds), nine of 32003 31 us,
// 128 of 152064 98 us (0.8 TB/s; 16.5, 28.8 and 54.5: vector ALU 51, 34 and 23 % of the time, LDS conflicts of the bins' atomics,
// and a row's sort and choice, one workgroup's chain).
// More collected tokens than fit (as where most logits are equal) are resolved by a radix selection over the row.
#include <algorithm>

#include "mmq_splitk.h"
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 1024;
constexpr int kBlock = 2048;                       // tokens whose masses are summed together
constexpr int kPer = kBlock / kThreads;
constexpr int kMaxBlocks = (1 << 20) / kBlock;
constexpr int kCap = 2048;                         // collected tokens
constexpr int kBatch = 256;                        // rows of a launch (at most 1024: a workgroup each)
constexpr double kLast = 30.498475;                // x beyond which rne(2^43 exp(-x)) is 0 (44 ln 2)
constexpr double kBinsPerX = 33.0;
static_assert(kLast * kBinsPerX < kBins, "bins");

// The scratch: what is zero between calls, then what has no initial value.
struct Zeroed {
    uint32_t count[kBatch][kBins];
    u64 mass[kBatch][kBins];
    uint32_t arrived[2][kBatch], collected[kBatch];
};
struct Cuts {
    int sure;                  // tokens of bins below this are kept
    int first, last, kbin;     // collected: bins first .. last (the cut of top-p), and kbin (that of top-k; -1: none)
    uint32_t k_left;           // tokens of kbin that top-k keeps
    u64 k_before, p_before;    // masses of the bins before kbin, before `first`
};
struct Free {
    u64 top[kBatch][kMaxBlocks];        // largest number of a workgroup's part
    Cuts cuts[kBatch];
    u64 list[kBatch][kCap];
    u64 block[kBatch][kMaxBlocks];      // masses
};
static_assert(sizeof(Zeroed) <= (4 << 20), "the zeroed part");

struct Args {
    Sample s;
    Zeroed* z;
    Free* f;
    int row0, parts, part_blocks;       // workgroups of a row, blocks of one
};

// Numbers in falling order of the logits, of equal ones the lower index above; 0 for a NaN and for -inf.
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t u = __builtin_bit_cast(uint32_t, l + 0.0f);   // -0 is 0
    return l > -__builtin_inff() ? (u >> 31 ? ~u : u | 0x80000000u) : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __builtin_bit_cast(float, key >> 31 ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ u64 number(float l, int i) {
    const uint32_t k = key_of(l);
    return k ? u64(k) << 32 | uint32_t(~i) : 0;
}

struct Smem {
    double two[64];            // 2^(j / 64)
    union {
        struct {
            uint32_t n[kBins];
            u64 w[kBins];
        } bins;
        u64 list[kCap];
    };
    u64 block[kMaxBlocks];
    u64 wave[2][2][kWaves];
    Cuts cuts;
    u64 cut, found, k_mass;
    uint32_t count, ticket;
    uint32_t key, above_n;
    u64 above_w;
};

struct Row {
    const float* l;
    int V;
    double top, inv;           // the largest logit, 1 / T
    double low;                // min_p
    u64 best;                  // the largest number
};

// x = (l_max - l) / T, 0 for the largest logit (also an infinity); not finite and never below 31 for a logit that does not count
__device__ __forceinline__ double distance(const Row& r, float l) {
    const double x = (r.top - double(l)) * r.inv;
    return double(l) == r.top ? 0.0 : x;
}
// e^-x and its mass, for 0 <= x <= kLast: 2^(n / 64) e^r, n = rne(-64 x / ln 2), e^r to r^5 / 120 (|r| < 0.0055).
__device__ __forceinline__ u64 weigh(const Smem& sm, double x, double& e) {
    constexpr double kMagic = 6755399441055744.0;                  // 2^52 + 2^51: the sum's low bits are the integer
    const double t = fma(x, -92.332482616893656877, kMagic);
    const int n = int(uint32_t(__builtin_bit_cast(u64, t)));
    const double nd = t - kMagic;
    double r = fma(nd, -0.010830424696249145458, -x);              // ln 2 / 64, and what its rounding left
    r = fma(nd, -3.623510646634843e-19, r);
    double p = fma(r, 1.0 / 120.0, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    e = ldexp(sm.two[n & 63] * p, n >> 6);
    return __builtin_bit_cast(u64, fma(e, 0x1p43, 0x1p52)) & ((u64(1) << 52) - 1);
}
__device__ __forceinline__ int bin_of(double x) { return int(x * kBinsPerX); }

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v) {    // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const u64 o = __shfl_up(v, off, 64);
        v += lane >= off ? o : 0;
    }
    return v;
}
// Sums of two numbers over the workgroup: inclusive up to each thread, and the totals.  Every thread calls; one barrier: calls
// that follow one another take turns with the two halves of sm.wave.
struct Sums {
    u64 a, b, all_a, all_b;
};
__device__ __forceinline__ Sums block_sums(Smem& sm, int turn, u64 a, u64 b = 0) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    a = wave_scan(a);
    b = wave_scan(b);
    if (lane == 63) {
        sm.wave[turn][0][wave] = a;
        sm.wave[turn][1][wave] = b;
    }
    __syncthreads();
    Sums s = {a, b, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const u64 x = sm.wave[turn][0][w], y = sm.wave[turn][1][w];
        s.all_a += x;
        s.all_b += y;
        s.a += w < wave ? x : 0;
        s.b += w < wave ? y : 0;
    }
    return s;
}

// f(block, i, l) for the row's tokens of blocks [b0, b1), kPer of a thread at a time (token j at i + j kThreads; behind the row's
// end l is a NaN), every thread of the workgroup in step; the loads of kAhead blocks are in flight together.
constexpr int kAhead = 4;
template <class F>
__device__ __forceinline__ void each(const Row& r, int b0, int b1, const F& f) {
    for (int b = b0; b < b1; b += kAhead) {
        float l[kAhead][kPer];
#pragma unroll
        for (int n = 0; n < kAhead; ++n)
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int i = (b + n) * kBlock + j * kThreads + threadIdx.x;
                l[n][j] = b + n < b1 && i < r.V ? r.l[i] : __builtin_nanf("");
            }
#pragma unroll
        for (int n = 0; n < kAhead; ++n)
            if (b + n < b1) f(b + n, (b + n) * kBlock + int(threadIdx.x), l[n]);
    }
}
// True where none of the wave's tokens reaches `floor`: nothing to do for them.
__device__ __forceinline__ bool all_below(const float (&l)[kPer], float floor) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) any |= l[j] >= floor;
    return __ballot(any) == 0;
}
// A logit that no token of distance up to x falls below.
__device__ __forceinline__ float floor_of(const Row& r, double T, double x) {
    const double f = r.top - x * T;
    const float low = float(f) - (fabsf(float(f)) + fabsf(float(r.top))) * 1e-6f;      // (more than the roundings of the terms)
    return low == low ? low : -__builtin_inff();                                     // (an infinite l_max)
}
// Masses by block: f(i, l, w) gives the tokens'; sums to sm.block[block].
template <class F>
__device__ __forceinline__ void sum_blocks(const Row& r, Smem& sm, int b0, int b1, float floor, const F& f) {
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads) sm.block[b] = 0;
    __syncthreads();
    each(r, b0, b1, [&](int block, int i, const float (&l)[kPer]) {
        if (all_below(l, floor)) return;
        u64 w[kPer], sum = 0;
        f(i, l, w);
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += w[j];
        sum = wave_sum(sum);
        if ((threadIdx.x & 63) == 0 && sum) atomicAdd(&sm.block[block], sum);
    });
    __syncthreads();
}

__device__ u64 pass_top(const Row& r, Smem& sm, int b0, int b1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 best = 0;
    each(r, b0, b1, [&](int, int i, const float (&l)[kPer]) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const u64 n = number(l[j], i + j * kThreads);
            best = n > best ? n : best;
        }
    });
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const u64 o = __shfl_xor(best, off, 64);
        best = o > best ? o : best;
    }
    if (lane == 0) sm.wave[0][0][wave] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = sm.wave[0][0][w] > best ? sm.wave[0][0][w] : best;
    return best;
}

// The row's settings, and whether there is a choice to make: else (greedy, or no token at all) `best` is the answer.
struct Settings {
    float T, p, low, u;
    int k;
    __device__ __forceinline__ Settings(const Args& a, int m)
        : T(a.s.temperature ? a.s.temperature[m] : 1.0f), p(a.s.top_p ? a.s.top_p[m] : 1.0f),
          low(a.s.min_p ? a.s.min_p[m] : 0.0f), u(a.s.u[m]), k(a.s.top_k ? a.s.top_k[m] : 0) {
        if (k < 0 || k >= a.s.V) k = 0;
        low = low < 1.0f ? low : low >= 1.0f ? 1.0f : 0.0f;   // (a NaN: none)
    }
    __device__ __forceinline__ bool chosen(u64 best) const { return best != 0 && T > 0.0f; }
    __device__ __forceinline__ bool cut() const { return k > 0 || p < 1.0f; }
};
__device__ __forceinline__ Row row_of(const Args& a, int m) { return {a.s.logits + m * a.s.stride, int(a.s.V)}; }
__device__ __forceinline__ void set_row(Row& r, const Settings& t, u64 best) {
    r.best = best;
    r.top = double(logit_of(uint32_t(best >> 32)));
    r.inv = 1.0 / double(t.T);
    r.low = double(t.low);
}
__device__ __forceinline__ void write_only(const Args& a, int m, u64 best) {
    if (threadIdx.x == 0) {
        a.s.ids[m] = best == 0 ? -1 : int(~uint32_t(best));
        if (a.s.probs) a.s.probs[m] = best == 0 ? 0.0f : 1.0f;
    }
}

__device__ void make_table(Smem& sm) {
    if (threadIdx.x < 64) sm.two[threadIdx.x] = exp2(double(threadIdx.x) / 64.0);
}

// Pass 2: this part's tokens into the bins of LDS.
__device__ void pass_bins(const Row& r, Smem& sm, bool masses, int b0, int b1) {
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
        sm.bins.n[b] = 0;
        sm.bins.w[b] = 0;
    }
    __syncthreads();
    const float floor = floor_of(r, 1.0 / r.inv, kLast);
    each(r, b0, b1, [&](int, int, const float (&l)[kPer]) {
        if (all_below(l, floor)) return;
        double x[kPer], e;
        u64 w[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[j] = distance(r, l[j]);
        if (masses)
#pragma unroll
            for (int j = 0; j < kPer; ++j) w[j] = weigh(sm, x[j] <= kLast ? x[j] : kLast, e);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (x[j] <= kLast) {
                const int b = bin_of(x[j]);
                atomicAdd(&sm.bins.n[b], 1u);
                if (masses) atomicAdd(&sm.bins.w[b], w[j]);
            }
    });
    __syncthreads();
}

// The cuts' bins, from the row's bins in LDS.
__device__ void find_bins(Smem& sm, int k, float p) {
    constexpr int kEach = kBins / kThreads;
    const int b0 = threadIdx.x * kEach;
    u64 n[kEach], w[kEach], n_sum = 0, w_sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        n[j] = sm.bins.n[b0 + j];
        w[j] = sm.bins.w[b0 + j];
        n_sum += n[j];
        w_sum += w[j];
    }
    if (threadIdx.x == 0) {
        sm.cuts = {kBins, kBins, -1, -1, 0, 0, 0};
        sm.k_mass = 0;
    }
    const Sums s = block_sums(sm, 0, n_sum, w_sum);
    // top-k's: the first bin at which the count reaches k
    const bool has_k = k > 0 && u64(k) < s.all_a;
    u64 nb = s.a - n_sum, wb = s.b - w_sum;
    if (has_k) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (nb < u64(k) && nb + n[j] >= u64(k)) {
                sm.cuts.kbin = sm.cuts.sure = b0 + j;
                sm.cuts.k_left = uint32_t(u64(k) - nb);
                sm.cuts.k_before = wb;
                sm.k_mass = w[j];
            }
            nb += n[j];
            wb += w[j];
        }
    } else if (threadIdx.x == 0) {
        sm.cuts.k_before = s.all_b;
    }
    __syncthreads();
    if (p < 1.0f) {
        // top-p's: its goal lies between those of the masses without and with all of kbin; the first bin whose sum reaches
        // it, at least the first that has a token: what is kept is never empty
        const u64 least = sm.cuts.k_before, most = least + sm.k_mass;
        const double lo = double(p) * double(least), hi = double(p) * double(most);
        wb = s.b - w_sum;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const u64 we = wb + w[j];
            if (we > 0 && double(we) >= lo && (wb == 0 || double(wb) < lo)) {
                sm.cuts.first = sm.cuts.sure = b0 + j;
                sm.cuts.p_before = wb;
            }
            if (we > 0 && double(we) >= hi && (wb == 0 || double(wb) < hi)) sm.cuts.last = b0 + j;
            wb = we;
        }
        __syncthreads();
    }
}

// Pass 3: masses of the part's blocks (sure tokens), and the tokens of the cuts' bins to sm.list, counted in sm.count (past
// kCap counted only).
__device__ void pass_masses(const Row& r, Smem& sm, const Cuts& c, int b0, int b1) {
    const int low_bin = max(max(c.sure - 1, c.last), c.kbin);          // (kBins - 1: all)
    sum_blocks(r, sm, b0, b1, floor_of(r, 1.0 / r.inv, min(kLast, (low_bin + 1) / kBinsPerX)), [&](int i, const float (&l)[kPer], u64 (&w)[kPer]) {
        double x[kPer];
        int bin[kPer];
        bool sure = false;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            x[j] = distance(r, l[j]);
            bin[j] = x[j] <= kLast ? bin_of(x[j]) : kBins;
            sure |= bin[j] < c.sure;
            w[j] = 0;
        }
        if (__ballot(sure) != 0)
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                double e;
                const u64 m = weigh(sm, bin[j] < kBins ? x[j] : kLast, e);
                w[j] = bin[j] < c.sure && (x[j] == 0.0 || e >= r.low) ? m : 0;
            }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if ((bin[j] >= c.first && bin[j] <= c.last) || bin[j] == c.kbin) {
                const uint32_t at = atomicAdd(&sm.count, 1u);
                if (at < kCap) sm.list[at] = number(l[j], i + j * kThreads);
            }
    });
}

// The collected numbers (n, in LDS) in falling order: each to its rank where a thread has one (the numbers differ), else sorted
// in a network.
__device__ void sort_list(Smem& sm, int n) {
    if (n <= kThreads) {
        const int i = threadIdx.x;
        const u64 mine = i < n ? sm.list[i] : 0;
        int rank = 0;
        if (i < ((n + 63) & ~63)) {
#pragma unroll 8
            for (int j = 0; j < n; ++j) rank += sm.list[j] > mine;
        }
        __syncthreads();
        if (i < n) sm.list[rank] = mine;
        __syncthreads();
        return;
    }
    int size = kThreads;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) sm.list[i] = 0;
    __syncthreads();
    for (int run = 2; run <= size; run <<= 1)
        for (int step = run >> 1; step; step >>= 1) {
            for (int i = threadIdx.x; i < size / 2; i += kThreads) {
                const int a = 2 * i - (i & (step - 1)), b = a + step;
                const u64 x = sm.list[a], y = sm.list[b];
                if ((x < y) == ((a & run) == 0)) {
                    sm.list[a] = y;
                    sm.list[b] = x;
                }
            }
            __syncthreads();
        }
}

// The cut from the sorted list; the kept tokens' masses go to their blocks.
__device__ void resolve_list(const Row& r, Smem& sm, int n, float p) {
    const Cuts c = sm.cuts;
    constexpr int kEach = kCap / kThreads;
    const int i0 = threadIdx.x * kEach;
    u64 number[kEach], w[kEach];
    double e[kEach];
    u64 ahead = 0, mass = 0;       // tokens before kbin (those of kbin are the list's last), masses of all
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        number[j] = i0 + j < n ? sm.list[i0 + j] : 0;
        w[j] = 0;
        if (number[j]) {
            const double x = distance(r, logit_of(uint32_t(number[j] >> 32)));
            w[j] = weigh(sm, x, e[j]);
            ahead += c.kbin < 0 || bin_of(x) < c.kbin;
        }
        mass += w[j];
    }
    if (threadIdx.x == 0) {
        sm.cut = ~u64(0);                             // (where the list keeps none: the sure ones alone)
        sm.k_mass = 0;
    }
    const Sums s = block_sums(sm, 0, mass, ahead);
    const int head = int(s.all_b), limit = c.kbin >= 0 ? min(n, head + int(c.k_left)) : n;      // of the list, by top-k
    u64 before = c.p_before + s.a - mass;
    if (p < 1.0f) {
        // mass of the first top_k: up to `limit`
        u64 at = s.a - mass, head_mass = 0, limit_mass = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (i0 + j == head) head_mass = at;
            if (i0 + j == limit) limit_mass = at;
            at += w[j];
        }
        // (each of one thread; a border at the list's end, or at the capacity's, is the sum of all)
        if (i0 <= head && head < i0 + kEach) sm.wave[1][0][0] = head_mass;
        if (i0 <= limit && limit < i0 + kEach) sm.wave[1][0][1] = limit_mass;
        __syncthreads();
        const u64 to_head = head < kCap ? sm.wave[1][0][0] : s.all_a, to_limit = limit < kCap ? sm.wave[1][0][1] : s.all_a;
        const double goal = double(p) * double(c.k_before + to_limit - to_head);
        // kept: those before which the sum has not reached the goal, and the first token.  (Between `last` and kbin the list
        // leaves tokens out: the sum has reached the goal there.)
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const u64 after = before + w[j];
            const bool in = i0 + j < limit && (before == 0 || double(before) < goal);
            if (in && (i0 + j + 1 >= limit || !(double(after) < goal))) sm.cut = number[j];
            before = after;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (i0 + j + 1 == limit) sm.cut = number[j];
    }
    __syncthreads();
    const u64 cut = sm.cut;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (number[j] && number[j] >= cut && (number[j] >> 32 == r.best >> 32 || e[j] >= r.low))
            atomicAdd(&sm.block[(~uint32_t(number[j])) / kBlock], w[j]);
    __syncthreads();
}

// The key at which a prefix ends, over the whole row by radix selection: by count (the limit-th token), or by mass (the first at
// which the sum reaches the goal).  above_n, above_w: tokens of larger keys.  floor: smaller numbers do not count.
__device__ void radix(const Row& r, Smem& sm, bool by_mass, double goal, u64 limit, u64 floor) {
    const int blocks = (r.V + kBlock - 1) / kBlock;
    if (threadIdx.x == 0) {
        sm.above_n = 0;
        sm.above_w = 0;
        sm.key = 0;
    }
    const int shifts[4] = {22, 12, 2, 0}, widths[4] = {10, 10, 10, 2};
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = shifts[pass], width = widths[pass], bins = 1 << width;
        for (int b = threadIdx.x; b < kBins; b += kThreads) {
            sm.bins.n[b] = 0;
            sm.bins.w[b] = 0;
        }
        __syncthreads();
        const uint32_t prefix = sm.key;
        each(r, 0, blocks, [&](int, int i, const float (&l)[kPer]) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const double x = distance(r, l[j]);
                const u64 n = number(l[j], i + j * kThreads);
                const uint32_t key = uint32_t(n >> 32);
                if (!(x <= kLast) || n < floor || (shift + width < 32 && key >> (shift + width) != prefix >> (shift + width))) continue;
                double e;
                atomicAdd(&sm.bins.n[(key >> shift) & (bins - 1)], 1u);
                atomicAdd(&sm.bins.w[(key >> shift) & (bins - 1)], weigh(sm, x, e));
            }
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t n = sm.above_n;
            u64 w = sm.above_w;
            int b = bins - 1, at = -1;
            uint32_t at_n = n;
            u64 at_w = w;
            for (; b >= 0; --b) {
                if (sm.bins.n[b] == 0) continue;
                at = b;
                at_n = n;
                at_w = w;
                if (by_mass ? double(w + sm.bins.w[b]) >= goal : n + sm.bins.n[b] >= limit) break;
                n += sm.bins.n[b];
                w += sm.bins.w[b];
            }
            sm.above_n = at_n;          // (never reached: every token is in, the cut is the lowest bin that has one)
            sm.above_w = at_w;
            sm.key = prefix | uint32_t(at < 0 ? 0 : at) << shift;
        }
        __syncthreads();
    }
}
// The number of the count-th token that has the key (the last one where there are fewer).
__device__ u64 nth(const Row& r, Smem& sm, uint32_t key, u64 count) {
    const int blocks = (r.V + kBlock - 1) / kBlock;
    if (threadIdx.x == 0) sm.found = 0;
    u64 seen = 0;
    for (int b = 0; b < blocks && seen < count; ++b) {
        // (kPer consecutive tokens a thread: index order)
        const int i0 = b * kBlock + threadIdx.x * kPer;
        u64 n = 0;
        for (int j = 0; j < kPer; ++j) n += i0 + j < r.V && key_of(r.l[i0 + j]) == key;
        const Sums s = block_sums(sm, b & 1, n);
        u64 at = seen + s.a - n;
        for (int j = 0; j < kPer; ++j)
            if (i0 + j < r.V && key_of(r.l[i0 + j]) == key) {
                ++at;
                if (at <= count) atomicMax(&sm.found, u64(i0 + j) + 1);
            }
        seen += s.all_a;
    }
    __syncthreads();
    const u64 i = sm.found;
    __syncthreads();
    return u64(key) << 32 | uint32_t(~uint32_t(i - 1));
}
__device__ void resolve_row(const Row& r, Smem& sm, int k, float p) {
    u64 cut = 1;
    if (k > 0) {
        radix(r, sm, false, 0.0, u64(k), 1);
        const uint32_t key = sm.key;
        const u64 left = u64(k) - min(u64(k), u64(sm.above_n));
        cut = nth(r, sm, key, left);
    }
    const int blocks = (r.V + kBlock - 1) / kBlock;
    if (p < 1.0f) {
        u64 w = 0;
        each(r, 0, blocks, [&](int, int i, const float (&l)[kPer]) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const double x = distance(r, l[j]);
                double e;
                if (x <= kLast && number(l[j], i + j * kThreads) >= cut) w += weigh(sm, x, e);
            }
        });
        const double goal = double(p) * double(block_sums(sm, 0, w).all_a);
        radix(r, sm, true, goal, 0, cut);
        const uint32_t key = sm.key;
        double e;
        const double each_w = double(weigh(sm, distance(r, logit_of(key)), e)), lack = goal - double(sm.above_w);
        const u64 n = lack > 0.0 && each_w > 0.0 ? u64(ceil(lack / each_w)) : 1;
        const u64 by_p = nth(r, sm, key, n);
        cut = by_p > cut ? by_p : cut;
    }
    __syncthreads();
    if (threadIdx.x == 0) sm.cut = cut;
    sum_blocks(r, sm, 0, blocks, -__builtin_inff(), [&](int i, const float (&l)[kPer], u64 (&w)[kPer]) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const double x = distance(r, l[j]);
            double e;
            w[j] = 0;
            if (!(x <= kLast) || number(l[j], i + j * kThreads) < cut) continue;
            const u64 m = weigh(sm, x, e);
            w[j] = x == 0.0 || e >= r.low ? m : 0;
        }
    });
}

// The choice: masses of the blocks in sm.block, kept are numbers from sm.cut on and those of bins below cuts.sure.
__device__ void choose(const Args& a, int m, const Row& r, Smem& sm, float u_row, bool by_bins) {
    const int blocks = (r.V + kBlock - 1) / kBlock;
    const u64 mine = int(threadIdx.x) < blocks ? sm.block[threadIdx.x] : 0;
    static_assert(kMaxBlocks <= kThreads, "a block a thread");
    const Sums s = block_sums(sm, 0, mine);
    const u64 total = s.all_a;
    const double u = u_row > 0.0f ? double(u_row) : 0.0;
    const u64 goal = u < 1.0 ? u64(floor(u * double(total))) : ~u64(0);
    const u64 need = goal < total - 1 ? goal : total - 1;   // the first token whose sum passes this
    if (mine != 0 && need < s.a && need >= s.a - mine) {
        sm.found = s.a - mine;
        sm.count = threadIdx.x;
    }
    __syncthreads();
    const int i0 = int(sm.count) * kBlock + threadIdx.x * kPer;
    float l[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) l[j] = i0 + j < r.V ? r.l[i0 + j] : __builtin_nanf("");
    u64 w[kPer], sum = 0;
    double e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const double x = distance(r, l[j]);
        w[j] = 0;
        e[j] = 0.0;
        if (x <= kLast && ((by_bins && bin_of(x) < sm.cuts.sure) || number(l[j], i0 + j) >= sm.cut)) {
            const u64 v = weigh(sm, x, e[j]);
            w[j] = x == 0.0 || e[j] >= r.low ? v : 0;
        }
        sum += w[j];
    }
    u64 at = sm.found + block_sums(sm, 1, sum).a - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (w[j] != 0 && at <= need && at + w[j] > need) {
            a.s.ids[m] = i0 + j;
            if (a.s.probs) a.s.probs[m] = float(e[j] / (double(total) * 0x1p-43));
        }
        at += w[j];
    }
}

__device__ void finish(const Args& a, int m, const Row& r, Smem& sm, const Settings& t, uint32_t collected) {
    if (collected > kCap) {
        resolve_row(r, sm, t.k, t.p);
        choose(a, m, r, sm, t.u, false);
        return;
    }
    if (sm.cuts.kbin >= 0 || t.p < 1.0f) {
        sort_list(sm, int(collected));
        resolve_list(r, sm, int(collected), t.p);
    } else {
        if (threadIdx.x == 0) sm.cut = ~u64(0);
        __syncthreads();
    }
    choose(a, m, r, sm, t.u, true);
}

// A workgroup per row, all passes.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(Args a) {
    __shared__ Smem sm;
    const int m = a.row0 + blockIdx.x, blocks = int((a.s.V + kBlock - 1) / kBlock);
    const Settings t(a, m);
    Row r = row_of(a, m);
    make_table(sm);
    const u64 best = pass_top(r, sm, 0, blocks);
    if (!t.chosen(best)) {
        write_only(a, m, best);
        return;
    }
    set_row(r, t, best);
    if (threadIdx.x == 0) {
        sm.cuts = {kBins, kBins, -1, -1, 0, 0, 0};
        sm.count = 0;
    }
    __syncthreads();
    if (t.cut()) {
        pass_bins(r, sm, t.p < 1.0f, 0, blocks);
        find_bins(sm, t.k, t.p);
    }
    const Cuts c = sm.cuts;
    pass_masses(r, sm, c, 0, blocks);
    finish(a, m, r, sm, t, sm.count);
}

// The passes as launches, a row over a.parts workgroups.
__global__ __launch_bounds__(kThreads) void sample_top_kernel(Args a) {
    __shared__ Smem sm;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, m = a.row0 + row;
    const int blocks = int((a.s.V + kBlock - 1) / kBlock);
    const u64 best = pass_top(row_of(a, m), sm, part * a.part_blocks, min(blocks, (part + 1) * a.part_blocks));
    if (threadIdx.x == 0) a.f->top[row][part] = best;
}
__device__ u64 row_top(const Args& a, int row) {
    const int lane = threadIdx.x & 63;
    u64 best = 0;
    for (int i = lane; i < a.parts; i += 64) {
        const u64 t = a.f->top[row][i];
        best = t > best ? t : best;
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const u64 o = __shfl_xor(best, off, 64);
        best = o > best ? o : best;
    }
    return best;
}
__global__ __launch_bounds__(kThreads) void sample_bins_kernel(Args a) {
    __shared__ Smem sm;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, m = a.row0 + row;
    const int blocks = int((a.s.V + kBlock - 1) / kBlock);
    const Settings t(a, m);
    const u64 best = row_top(a, row);
    if (!t.chosen(best) || !t.cut()) return;
    Row r = row_of(a, m);
    set_row(r, t, best);
    make_table(sm);
    pass_bins(r, sm, t.p < 1.0f, part * a.part_blocks, min(blocks, (part + 1) * a.part_blocks));
    for (int b = threadIdx.x; b < kBins; b += kThreads)
        if (sm.bins.n[b]) {
            __hip_atomic_fetch_add(&a.z->count[row][b], sm.bins.n[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (t.p < 1.0f) __hip_atomic_fetch_add(&a.z->mass[row][b], sm.bins.w[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    if (!splitk_arrive(&a.z->arrived[0][row], a.parts, &sm.ticket)) return;
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
        sm.bins.n[b] = __hip_atomic_load(&a.z->count[row][b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        sm.bins.w[b] = __hip_atomic_load(&a.z->mass[row][b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.z->count[row][b], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.z->mass[row][b], u64(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    find_bins(sm, t.k, t.p);
    __syncthreads();
    if (threadIdx.x == 0) a.f->cuts[row] = sm.cuts;
}
__global__ __launch_bounds__(kThreads) void sample_choose_kernel(Args a) {
    __shared__ Smem sm;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, m = a.row0 + row;
    const int blocks = int((a.s.V + kBlock - 1) / kBlock);
    const Settings t(a, m);
    const Cuts found = a.f->cuts[row];         // (not set where the row is not cut)
    const u64 best = row_top(a, row);
    if (!t.chosen(best)) {
        if (part == 0) write_only(a, m, best);
        return;
    }
    Row r = row_of(a, m);
    set_row(r, t, best);
    make_table(sm);
    const Cuts c = t.cut() ? found : Cuts{kBins, kBins, -1, -1, 0, 0, 0};
    if (threadIdx.x == 0) {
        sm.cuts = c;
        sm.count = 0;
    }
    const int b0 = part * a.part_blocks, b1 = min(blocks, (part + 1) * a.part_blocks);
    pass_masses(r, sm, c, b0, b1);
    for (int b = b0 + threadIdx.x; b < b1; b += kThreads)
        __hip_atomic_store(&a.f->block[row][b], sm.block[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t mine = sm.count;
    if (mine) {       // (the same on every thread)
        if (threadIdx.x == 0)
            sm.ticket = __hip_atomic_fetch_add(&a.z->collected[row], mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const uint32_t at = sm.ticket;
        for (uint32_t i = threadIdx.x; i < min(mine, uint32_t(kCap)) && at + i < kCap; i += kThreads)
            __hip_atomic_store(&a.f->list[row][at + i], sm.list[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (!splitk_arrive(&a.z->arrived[1][row], a.parts, &sm.ticket)) return;
    // (the whole list's places are loaded: how many count is known no earlier)
    const uint32_t collected = __hip_atomic_load(&a.z->collected[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    u64 part_list[kCap / kThreads];
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j)
        part_list[j] = __hip_atomic_load(&a.f->list[row][j * kThreads + threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (int(threadIdx.x) < blocks)
        sm.block[threadIdx.x] = __hip_atomic_load(&a.f->block[row][threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int j = 0; j < kCap / kThreads; ++j) sm.list[j * kThreads + threadIdx.x] = part_list[j];
    __syncthreads();
    if (threadIdx.x == 0) __hip_atomic_store(&a.z->collected[row], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    finish(a, m, r, sm, t, collected);
}

}  // namespace

// (the same for every size: one buffer serves calls of any)
size_t sample_scratch_bytes(int64_t, int64_t) { return (size_t(4) << 20) + sizeof(Free); }

hipError_t launch_sample(const Sample& r, hipStream_t s, const char** name) {
    Args a;
    a.s = r;
    a.z = static_cast<Zeroed*>(r.scratch);
    a.f = reinterpret_cast<Free*>(static_cast<uint8_t*>(r.scratch) + (size_t(4) << 20));
    const int blocks = int((r.V + kBlock - 1) / kBlock);
    for (int64_t m = 0; m < r.M; m += kBatch) {
        const int rows = int(std::min<int64_t>(kBatch, r.M - m));
        a.row0 = int(m);
        // about four workgroups a CU; rows of one or two blocks are left whole.  One row, and 256, with top-k and top-p, in us, whole
        // and in launches: 4096 tokens 15 and 16, 21 and 29; 8192 17 and 19, 21 and 52 (the rule's loss, as for 128 rows
        // to about 32000: 38, 53); 16384 25 and 26, 22 and 55; 152064 111 and 129, 25 and 127
        a.parts = blocks <= 2 ? 1 : std::min(blocks, 1024 / rows);
        a.part_blocks = (blocks + a.parts - 1) / a.parts;
        a.parts = (blocks + a.part_blocks - 1) / a.part_blocks;
        if (a.parts == 1) {
            *name = "sample_row";
            hipLaunchKernelGGL(sample_row_kernel, dim3(rows), dim3(kThreads), 0, s, a);
        } else {
            *name = "sample";
            const dim3 grid(unsigned(rows) * unsigned(a.parts));
            hipLaunchKernelGGL(sample_top_kernel, grid, dim3(kThreads), 0, s, a);
            if (r.top_k || r.top_p) hipLaunchKernelGGL(sample_bins_kernel, grid, dim3(kThreads), 0, s, a);
            hipLaunchKernelGGL(sample_choose_kernel, grid, dim3(kThreads), 0, s, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace mq
