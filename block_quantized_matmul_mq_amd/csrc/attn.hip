// mq_attn: attention over the paged cache of keys and values in blocks of 4 or 8 bits.
//
//   O[t][h] = sum_j softmax_j(scale Q[t][h] . K[j]) V[j],  head h reads the cache's head h / (q_heads / heads),
//   over the keys j that token t sees; a token that sees none gets zeros.
#include "kv_layout.h"
#include "mq_device.h"
#include "mq_internal.h"

namespace mq {

namespace {

constexpr int kThreads = 256;

struct AttnArgs {
    KvView c;
    const float* q;
    float* out;
    int64_t q_stride;
    int q_heads, causal, window, max_q, max_kv;
    float scale;
};

// A workgroup per query row; a thread per key of a chunk for the scores, per dimension for the sums.
template <int BITS, int D>
__global__ __launch_bounds__(kThreads) void attn_kernel(AttnArgs a) {
    using L = KvLayout<BITS, D>;
    __shared__ float qs[D], p[kThreads], red[kThreads / 64];
    __shared__ int where[kThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t = blockIdx.x, h = blockIdx.y, kvh = h / (a.q_heads / a.c.heads);
    const KvToken tok = kv_token(a.c, t);
    if (tok.seq < 0) return;
    if (t - a.c.q_start[tok.seq] >= a.max_q) return;
    const int len = min(a.c.kv_len[tok.seq], a.max_kv);
    const int end = a.causal ? min(len, tok.pos + 1) : len;
    const int begin = a.window > 0 ? max(0, tok.pos + 1 - a.window) : 0;
    if (tid < D) qs[tid] = a.q[t * a.q_stride + int64_t(h) * D + tid];
    const int64_t section = int64_t(a.c.page_tokens) * L::kRow;
    float m = -__builtin_inff(), l = 0.0f, o = 0.0f;
    for (int j0 = begin; j0 < end; j0 += kThreads) {
        const int j = j0 + tid;
        const int page = j < end ? kv_page(a.c, tok.seq, j) : -1;
        const int slot = j & (a.c.page_tokens - 1);
        __syncthreads();
        where[tid] = page;
        float s = -__builtin_inff();
        if (page >= 0) {
            const uint8_t* chunk = a.c.data + (int64_t(page) * a.c.heads + kvh) * a.c.chunk;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(chunk + 2 * section) + int64_t(slot) * L::kBlocks;
            s = 0.0f;
            for (int d = 0; d < D; ++d) {
                int code = chunk[L::k_byte(slot, d)];
                if constexpr (BITS == 4) code = (code >> (4 * L::k_nibble(d))) & 15;
                s = fmaf(qs[d], float(code - L::kOffset) * half_bits_to_float(scales[d / 32]), s);
            }
            s *= a.scale;
        }
        float top = s;
        for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        if (lane == 0) red[wave] = top;
        __syncthreads();
        top = m;
        for (int w = 0; w < kThreads / 64; ++w) top = fmaxf(top, red[w]);
        const float keep = m == top ? 1.0f : expf(m - top);
        p[tid] = page < 0 ? 0.0f : expf(s - top);
        m = top;
        __syncthreads();
        l *= keep;
        o *= keep;
        for (int i = 0; i < kThreads; ++i) {
            if (where[i] < 0) continue;
            l += p[i];
            if (tid < D) {
                const uint8_t* chunk = a.c.data + (int64_t(where[i]) * a.c.heads + kvh) * a.c.chunk;
                const int sl = (j0 + i) & (a.c.page_tokens - 1);
                const uint16_t* scales = reinterpret_cast<const uint16_t*>(chunk + 2 * section) +
                                         int64_t(a.c.page_tokens + sl) * L::kBlocks;
                int code = chunk[section + L::v_byte(sl, tid)];
                if constexpr (BITS == 4) code = (code >> (4 * L::v_nibble(tid))) & 15;
                o = fmaf(p[i], float(code - L::kOffset) * half_bits_to_float(scales[tid / 32]), o);
            }
        }
    }
    if (tid < D) a.out[(int64_t(t) * a.q_heads + h) * D + tid] = l == 0.0f ? 0.0f : o / l;
}

}  // namespace

size_t attn_scratch_bytes(int, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attn(const Attn& r, hipStream_t s, const char** name) {
    *name = "attn";
    const AttnArgs a = {r.cache.view, r.q, r.out, r.q_stride, int(r.q_heads), r.causal, int(r.window), int(r.max_q), int(r.max_kv), r.scale};
    const dim3 grid(unsigned(r.T), unsigned(r.q_heads));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a); };
    const int64_t d = r.cache.dim;
    if (r.cache.bits == 4) d == 64 ? run(attn_kernel<4, 64>) : d == 128 ? run(attn_kernel<4, 128>) : run(attn_kernel<4, 256>);
    else d == 64 ? run(attn_kernel<8, 64>) : d == 128 ? run(attn_kernel<8, 128>) : run(attn_kernel<8, 256>);
    return hipGetLastError();
}

}  // namespace mq
