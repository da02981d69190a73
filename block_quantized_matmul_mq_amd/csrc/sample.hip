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
// A row is divided over workgroups and the passes over launches (the last workgroup of a row does a pass's single
// part, mmq_splitk.h's exchange) where that is faster than a workgroup that makes all passes of a row by itself.
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
constexpr int kBatch = 256;                        // rows of a launch
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
    u64 wave_a[kWaves], wave_b[kWaves];
    Cuts cuts;
    u64 cut, total, found;
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
// Inclusive sums over the workgroup's threads; every thread calls, red is free again afterwards.
__device__ u64 block_scan(u64 v, u64* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_scan(v);
    if (lane == 63) red[wave] = v;
    __syncthreads();
    for (int w = 0; w < wave; ++w) v += red[w];
    __syncthreads();
    return v;
}
__device__ u64 block_sum(u64 v, u64* red) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    v = wave_sum(v);
    if (lane == 0) red[wave] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kWaves; ++w) v += red[w];
    __syncthreads();
    return v;
}

// f(i, l) for the row's tokens of blocks [b0, b1), every thread of the workgroup in step (i >= V: l is a NaN).
template <class F>
__device__ __forceinline__ void each(const Row& r, int b0, int b1, const F& f) {
    for (int b = b0; b < b1; ++b) {
        float l[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = b * kBlock + j * kThreads + threadIdx.x;
            l[j] = i < r.V ? r.l[i] : __builtin_nanf("");
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) f(b * kBlock + j * kThreads + int(threadIdx.x), l[j]);
    }
}

__device__ u64 pass_top(const Row& r, Smem& sm, int b0, int b1) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 best = 0;
    each(r, b0, b1, [&](int i, float l) {
        const u64 n = number(l, i);
        best = n > best ? n : best;
    });
#pragma unroll
    for (int off = 32; off; off >>= 1) {
        const u64 o = __shfl_xor(best, off, 64);
        best = o > best ? o : best;
    }
    if (lane == 0) sm.wave_a[wave] = best;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) best = sm.wave_a[w] > best ? sm.wave_a[w] : best;
    __syncthreads();
    return best;
}

// The row's settings.  True where there is a choice to make: else (greedy, or no token at all) `best` is the answer.
__device__ __forceinline__ bool settings(const Args& a, int m, u64 best, Row& r, int& k, float& p) {
    const float T = a.s.temperature ? a.s.temperature[m] : 1.0f;
    r.best = best;
    if (best == 0 || !(T > 0.0f)) return false;
    r.top = double(logit_of(uint32_t(best >> 32)));
    r.inv = 1.0 / double(T);
    k = a.s.top_k ? a.s.top_k[m] : 0;
    k = k > 0 && k < r.V ? k : 0;
    p = a.s.top_p ? a.s.top_p[m] : 1.0f;
    const float mp = a.s.min_p ? a.s.min_p[m] : 0.0f;
    r.low = mp < 1.0f ? double(mp) : mp >= 1.0f ? 1.0 : 0.0;   // (a NaN: none)
    return true;
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
    each(r, b0, b1, [&](int, float l) {
        const double x = distance(r, l);
        if (!(x <= kLast)) return;
        const int b = bin_of(x);
        atomicAdd(&sm.bins.n[b], 1u);
        if (masses) {
            double e;
            atomicAdd(&sm.bins.w[b], weigh(sm, x, e));
        }
    });
    __syncthreads();
}

// The cuts' bins, from the row's bins in LDS.
__device__ void find_bins(Smem& sm, int k, float p) {
    constexpr int kEach = kBins / kThreads;
    const int b0 = threadIdx.x * kEach;
    u64 n = 0, w = 0;
    for (int j = 0; j < kEach; ++j) {
        n += sm.bins.n[b0 + j];
        w += sm.bins.w[b0 + j];
    }
    u64 n_before = block_scan(n, sm.wave_a) - n, w_before = block_scan(w, sm.wave_b) - w;
    const u64 all_n = block_sum(n, sm.wave_a), all_w = block_sum(w, sm.wave_b);
    if (threadIdx.x == 0) sm.cuts = {kBins, kBins, -1, -1, 0, all_w, 0};
    __syncthreads();
    // top-k's: the first bin at which the count reaches k
    if (k > 0 && u64(k) < all_n) {
        u64 nb = n_before, wb = w_before;
        for (int j = 0; j < kEach; ++j) {
            if (nb < u64(k) && nb + sm.bins.n[b0 + j] >= u64(k)) {
                sm.cuts.kbin = sm.cuts.sure = b0 + j;
                sm.cuts.k_left = uint32_t(u64(k) - nb);
                sm.cuts.k_before = wb;
            }
            nb += sm.bins.n[b0 + j];
            wb += sm.bins.w[b0 + j];
        }
    }
    __syncthreads();
    if (p < 1.0f) {
        // top-p's: its goal lies between those of the masses without and with all of kbin
        const u64 most = sm.cuts.kbin < 0 ? all_w : sm.cuts.k_before + sm.bins.w[sm.cuts.kbin];
        const double lo = double(p) * double(sm.cuts.k_before), hi = double(p) * double(most);
        // (the first bin whose sum reaches a goal; at least the first that has a token: what is kept is never empty)
        u64 wb = w_before;
        for (int j = 0; j < kEach; ++j) {
            const u64 we = wb + sm.bins.w[b0 + j];
            if (we > 0 && double(we) >= lo && (wb == 0 || double(wb) < lo)) {
                sm.cuts.first = b0 + j;
                sm.cuts.p_before = wb;
            }
            if (we > 0 && double(we) >= hi && (wb == 0 || double(wb) < hi)) sm.cuts.last = b0 + j;
            wb = we;
        }
        __syncthreads();
        if (threadIdx.x == 0) sm.cuts.sure = sm.cuts.first;
    }
    __syncthreads();
}

// Pass 3: masses of the part's blocks (sure tokens) and the tokens of the cuts' bins.
template <class Put, class Block>
__device__ __forceinline__ void pass_masses(const Row& r, Smem& sm, const Cuts& c, int b0, int b1, const Put& put, const Block& block) {
    for (int b = b0; b < b1; ++b) {
        u64 w = 0;
        each(r, b, b + 1, [&](int i, float l) {
            const double x = distance(r, l);
            if (!(x <= kLast)) return;
            const int bin = bin_of(x);
            if (bin < c.sure) {
                double e;
                const u64 m = weigh(sm, x, e);
                w += x == 0.0 || e >= r.low ? m : 0;
            }
            if ((bin >= c.first && bin <= c.last) || bin == c.kbin) put(number(l, i));
        });
        w = block_sum(w, sm.wave_a);
        if (threadIdx.x == 0) block(b, w);
    }
}

// The collected numbers (n, in LDS) in falling order.
__device__ void sort_list(Smem& sm, int n) {
    int size = 64;
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

__device__ __forceinline__ u64 weigh_number(const Row& r, const Smem& sm, u64 number, double& e) {
    const double x = distance(r, logit_of(uint32_t(number >> 32)));
    return weigh(sm, x, e);
}

// The cut from the sorted list; the kept tokens' masses go to their blocks.
__device__ void resolve_list(const Row& r, Smem& sm, int n, float p) {
    const Cuts c = sm.cuts;
    constexpr int kEach = kCap / kThreads;
    const int i0 = threadIdx.x * kEach;
    // tokens of kbin are the last of the list where there is one; `head` of the list are before them
    u64 in_head = 0;
    for (int j = 0; j < kEach; ++j)
        if (i0 + j < n && c.kbin >= 0) in_head += bin_of(distance(r, logit_of(uint32_t(sm.list[i0 + j] >> 32)))) < c.kbin;
    const int head = c.kbin >= 0 ? int(block_sum(in_head, sm.wave_a)) : n;
    const int limit = c.kbin >= 0 ? min(n, head + int(c.k_left)) : n;      // of the list, by top-k
    if (p < 1.0f) {
        u64 w[kEach], mine = 0, mine_k = 0;
        for (int j = 0; j < kEach; ++j) {
            double e;
            w[j] = i0 + j < limit ? weigh_number(r, sm, sm.list[i0 + j], e) : 0;
            mine += w[j];
            if (i0 + j >= head) mine_k += w[j];
        }
        const u64 whole = c.k_before + block_sum(mine_k, sm.wave_a);       // mass of the first top_k
        const double goal = double(p) * double(whole);
        u64 before = c.p_before + block_scan(mine, sm.wave_b) - mine;
        if (threadIdx.x == 0) sm.cut = c.p_before == 0 ? r.best : 0;       // (at least the first token)
        __syncthreads();
        // kept: those before which the sum has not reached the goal.  (Between `last` and kbin the list leaves tokens out: the
        // sum has reached the goal there.)
        u64 last = 0;
        for (int j = 0; j < kEach; ++j) {
            if (i0 + j < limit && double(before) < goal) last = sm.list[i0 + j];
            before += w[j];
        }
        const u64 who = __ballot(last != 0);
        // the smallest number kept: of the last wave that has one (numbers fall along the list)
        if (who) {
            const u64 v = __shfl(last, 63 - __clzll(who), 64);
            if ((threadIdx.x & 63) == 0) sm.wave_a[threadIdx.x >> 6] = v;
        } else if ((threadIdx.x & 63) == 0) {
            sm.wave_a[threadIdx.x >> 6] = 0;
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int v = 0; v < kWaves; ++v)
                if (sm.wave_a[v]) sm.cut = sm.wave_a[v];
        __syncthreads();
        if (threadIdx.x == 0 && sm.cut == 0) sm.cut = ~u64(0);             // (none of the list: the sure ones alone)
    } else if (threadIdx.x == 0) {
        sm.cut = limit > 0 ? sm.list[limit - 1] : 0;
    }
    __syncthreads();
    for (int j = 0; j < kEach; ++j) {
        if (i0 + j >= n || sm.list[i0 + j] < sm.cut) continue;
        double e;
        const u64 m = weigh_number(r, sm, sm.list[i0 + j], e);
        if (sm.list[i0 + j] >> 32 == r.best >> 32 || e >= r.low) atomicAdd(&sm.block[(~uint32_t(sm.list[i0 + j])) / kBlock], m);
    }
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
        each(r, 0, blocks, [&](int i, float l) {
            const double x = distance(r, l);
            const u64 n = number(l, i);
            const uint32_t key = uint32_t(n >> 32);
            if (!(x <= kLast) || n < floor || (shift + width < 32 && key >> (shift + width) != prefix >> (shift + width))) return;
            double e;
            atomicAdd(&sm.bins.n[(key >> shift) & (bins - 1)], 1u);
            atomicAdd(&sm.bins.w[(key >> shift) & (bins - 1)], weigh(sm, x, e));
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
    __syncthreads();
    u64 seen = 0;
    for (int b = 0; b < blocks; ++b) {
        // (kPer consecutive tokens a thread: index order)
        const int i0 = b * kBlock + threadIdx.x * kPer;
        u64 n = 0;
        for (int j = 0; j < kPer; ++j) n += i0 + j < r.V && key_of(r.l[i0 + j]) == key;
        const u64 upto = seen + block_scan(n, sm.wave_a);
        u64 at = upto - n;
        for (int j = 0; j < kPer; ++j)
            if (i0 + j < r.V && key_of(r.l[i0 + j]) == key) {
                ++at;
                if (at <= count) atomicMax(reinterpret_cast<unsigned long long*>(&sm.found), u64(i0 + j) + 1);
            }
        seen += block_sum(n, sm.wave_b);
        if (seen >= count) break;
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
        each(r, 0, blocks, [&](int i, float l) {
            const double x = distance(r, l);
            double e;
            if (x <= kLast && number(l, i) >= cut) w += weigh(sm, x, e);
        });
        const double goal = double(p) * double(block_sum(w, sm.wave_a));
        radix(r, sm, true, goal, 0, cut);
        const uint32_t key = sm.key;
        double e;
        const double each_w = double(weigh_number(r, sm, u64(key) << 32, e)), lack = goal - double(sm.above_w);
        const u64 n = lack > 0.0 && each_w > 0.0 ? u64(ceil(lack / each_w)) : 1;
        const u64 by_p = nth(r, sm, key, n);
        cut = by_p > cut ? by_p : cut;
    }
    __syncthreads();
    if (threadIdx.x == 0) sm.cut = cut;
    for (int b = 0; b < blocks; ++b) {
        u64 w = 0;
        each(r, b, b + 1, [&](int i, float l) {
            const double x = distance(r, l);
            if (!(x <= kLast) || number(l, i) < cut) return;
            double e;
            const u64 m = weigh(sm, x, e);
            w += x == 0.0 || e >= r.low ? m : 0;
        });
        w = block_sum(w, sm.wave_a);
        if (threadIdx.x == 0) sm.block[b] = w;
    }
    __syncthreads();
}

// The choice: masses of the blocks in sm.block, kept are numbers from sm.cut on and those of bins below cuts.sure.
__device__ void choose(const Args& a, int m, const Row& r, Smem& sm, bool by_bins) {
    const int blocks = (r.V + kBlock - 1) / kBlock;
    const u64 mine = int(threadIdx.x) < blocks ? sm.block[threadIdx.x] : 0;
    static_assert(kMaxBlocks <= kThreads, "a block a thread");
    const u64 upto = block_scan(mine, sm.wave_a);
    const u64 total = block_sum(mine, sm.wave_b);
    double u = double(a.s.u[m]);
    u = u > 0.0 ? u : 0.0;
    const u64 goal = u < 1.0 ? u64(floor(u * double(total))) : ~u64(0);
    const u64 need = goal < total - 1 ? goal : total - 1;   // the first token whose sum passes this
    if (mine != 0 && need < upto && need >= upto - mine) {
        sm.found = upto - mine;
        sm.count = threadIdx.x;
    }
    __syncthreads();
    const int i0 = int(sm.count) * kBlock + threadIdx.x * kPer;
    u64 w[kPer], sum = 0;
    double e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = i0 + j;
        const float l = i < r.V ? r.l[i] : __builtin_nanf("");
        const double x = distance(r, l);
        w[j] = 0;
        e[j] = 0.0;
        if (x <= kLast && ((by_bins && bin_of(x) < sm.cuts.sure) || number(l, i) >= sm.cut)) {
            const u64 v = weigh(sm, x, e[j]);
            w[j] = x == 0.0 || e[j] >= r.low ? v : 0;
        }
        sum += w[j];
    }
    u64 at = sm.found + block_scan(sum, sm.wave_a) - sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (w[j] != 0 && at <= need && at + w[j] > need) {
            a.s.ids[m] = i0 + j;
            if (a.s.probs) a.s.probs[m] = float(e[j] / (double(total) * 0x1p-43));
        }
        at += w[j];
    }
}

__device__ void finish(const Args& a, int m, const Row& r, Smem& sm, int k, float p, uint32_t collected) {
    if (collected > kCap) {
        resolve_row(r, sm, k, p);
        choose(a, m, r, sm, false);
        return;
    }
    if (sm.cuts.kbin >= 0 || p < 1.0f) {
        sort_list(sm, int(collected));
        resolve_list(r, sm, int(collected), p);
    } else if (threadIdx.x == 0) {
        sm.cut = ~u64(0);
    }
    __syncthreads();
    choose(a, m, r, sm, true);
}

// A workgroup per row, all passes.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(Args a) {
    __shared__ Smem sm;
    const int m = a.row0 + blockIdx.x, blocks = int((a.s.V + kBlock - 1) / kBlock);
    Row r = {a.s.logits + m * a.s.stride, int(a.s.V)};
    make_table(sm);
    const u64 best = pass_top(r, sm, 0, blocks);
    int k;
    float p;
    if (!settings(a, m, best, r, k, p)) {
        write_only(a, m, best);
        return;
    }
    if (threadIdx.x == 0) {
        sm.cuts = {kBins, kBins, -1, -1, 0, 0, 0};
        sm.count = 0;
    }
    __syncthreads();
    if (k > 0 || p < 1.0f) {
        pass_bins(r, sm, p < 1.0f, 0, blocks);
        find_bins(sm, k, p);
    }
    const Cuts c = sm.cuts;
    pass_masses(r, sm, c, 0, blocks,
                [&](u64 n) {
                    const uint32_t at = atomicAdd(&sm.count, 1u);
                    if (at < kCap) sm.list[at] = n;
                },
                [&](int b, u64 w) { sm.block[b] = w; });
    __syncthreads();
    const uint32_t collected = sm.count;
    __syncthreads();
    finish(a, m, r, sm, k, p, collected);
}

// The passes as launches, a row over a.parts workgroups.
__global__ __launch_bounds__(kThreads) void sample_top_kernel(Args a) {
    __shared__ Smem sm;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, m = a.row0 + row;
    const int blocks = int((a.s.V + kBlock - 1) / kBlock);
    const Row r = {a.s.logits + m * a.s.stride, int(a.s.V)};
    const u64 best = pass_top(r, sm, part * a.part_blocks, min(blocks, (part + 1) * a.part_blocks));
    if (threadIdx.x == 0) a.f->top[row][part] = best;
}
__device__ u64 row_top(const Args& a, Smem& sm, int row) {
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
    Row r = {a.s.logits + m * a.s.stride, int(a.s.V)};
    int k;
    float p;
    if (!settings(a, m, row_top(a, sm, row), r, k, p) || (k == 0 && !(p < 1.0f))) return;
    make_table(sm);
    __syncthreads();
    pass_bins(r, sm, p < 1.0f, part * a.part_blocks, min(blocks, (part + 1) * a.part_blocks));
    for (int b = threadIdx.x; b < kBins; b += kThreads)
        if (sm.bins.n[b]) {
            __hip_atomic_fetch_add(&a.z->count[row][b], sm.bins.n[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (p < 1.0f) __hip_atomic_fetch_add(&a.z->mass[row][b], sm.bins.w[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    if (!splitk_arrive(&a.z->arrived[0][row], a.parts, &sm.ticket)) return;
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
        sm.bins.n[b] = __hip_atomic_load(&a.z->count[row][b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        sm.bins.w[b] = __hip_atomic_load(&a.z->mass[row][b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.z->count[row][b], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&a.z->mass[row][b], u64(0), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    find_bins(sm, k, p);
    if (threadIdx.x == 0) a.f->cuts[row] = sm.cuts;
}
__global__ __launch_bounds__(kThreads) void sample_choose_kernel(Args a) {
    __shared__ Smem sm;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts, m = a.row0 + row;
    const int blocks = int((a.s.V + kBlock - 1) / kBlock);
    Row r = {a.s.logits + m * a.s.stride, int(a.s.V)};
    int k;
    float p;
    const u64 best = row_top(a, sm, row);
    if (!settings(a, m, best, r, k, p)) {
        if (part == 0) write_only(a, m, best);
        return;
    }
    make_table(sm);
    if (threadIdx.x == 0) {
        sm.cuts = {kBins, kBins, -1, -1, 0, 0, 0};
        if (k > 0 || p < 1.0f) sm.cuts = a.f->cuts[row];
    }
    __syncthreads();
    const Cuts c = sm.cuts;
    pass_masses(r, sm, c, part * a.part_blocks, min(blocks, (part + 1) * a.part_blocks),
                [&](u64 n) {
                    const uint32_t at = __hip_atomic_fetch_add(&a.z->collected[row], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                    if (at < kCap) __hip_atomic_store(&a.f->list[row][at], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                },
                [&](int b, u64 w) { __hip_atomic_store(&a.f->block[row][b], w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); });
    if (!splitk_arrive(&a.z->arrived[1][row], a.parts, &sm.ticket)) return;
    const uint32_t collected = __hip_atomic_load(&a.z->collected[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = threadIdx.x; i < int(min(collected, uint32_t(kCap))); i += kThreads)
        sm.list[i] = __hip_atomic_load(&a.f->list[row][i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = threadIdx.x; i < blocks; i += kThreads)
        sm.block[i] = __hip_atomic_load(&a.f->block[row][i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (threadIdx.x == 0) __hip_atomic_store(&a.z->collected[row], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    finish(a, m, r, sm, k, p, collected);
}

}  // namespace

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
        // about two workgroups a CU; rows enough for that, or short ones, are left whole
        a.parts = std::min(blocks, std::max(1, 512 / rows));
        if (a.parts <= 2) a.parts = rows >= 128 ? a.parts : 1;
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
