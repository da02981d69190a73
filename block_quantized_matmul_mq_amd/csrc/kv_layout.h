// The paged cache of keys and values (mq_kv_append, mq_kv_read, mq_attn): byte layout and lookups.
//
// A page holds P tokens of every head; page p's chunk of head h starts at (p heads + h) chunk bytes and
// holds four sections, of P tokens each:
//   K codes, V codes   P D bits / 8 bytes each
//   K scales, V scales f16 [P][D / 32] each
// A block is 32 consecutive dimensions of one token: value = d (code - offset), codes of 4 bits (offset 8)
// or 8 bits (offset 128).  Inside the code sections the order is the one in which the matrix units take
// them (attn.hip): a lane's operand is one dword or a few, and a wave's 64 lanes read 16 tokens as one
// contiguous run.  With NB = D / 32:
//   K  token t's row of D bits / 8 bytes: dimension 32 b + 8 g + n (g = 0..3, n = 0..7) is the n-th code
//      of the (bits)-byte unit g NB + b (low nibble first).
//   V  16-token tile t / 16, then lane (t % 16 / 4, c = dim % 16), token pair t % 4 / 2, unit i, token
//      parity t % 2: two bytes, the codes of dimensions c + 16 j of the i-th run of 64 dimensions
//      (4 bits: j = 0..3, low nibble first) or of 32 (8 bits: j = 0, 1).
// Two tokens never share a byte, so tokens are appended without reading their neighbours.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

namespace mq {

// Sequences of a call: sequence b's tokens are rows q_start[b] .. q_start[b + 1] - 1 and its cache holds
// kv_len[b] tokens with them, token j in page table[b][j / P] at j % P.
struct KvView {
    uint8_t* data;
    const int32_t *q_start, *kv_len, *table;
    int64_t chunk;           // bytes of a page's chunk of one head
    int pages, page_tokens, page_shift, heads, seqs, width;
};

template <int BITS, int D>
struct KvLayout {
    static constexpr int kBlocks = D / 32;
    static constexpr int kRow = D * BITS / 8;             // code bytes of a token
    static constexpr int kOffset = BITS == 4 ? 8 : 128;
    static constexpr int kUnitDims = 256 / BITS;          // dimensions that a V unit and its 15 neighbours cover
    static constexpr int kUnits = D / kUnitDims;
    // byte (and for 4 bits nibble) of dimension `dim` of token t in a code section
    static __host__ __device__ constexpr int64_t k_byte(int t, int dim) {
        return int64_t(t) * kRow + (dim % 32 / 8 * kBlocks + dim / 32) * BITS + dim % 8 * BITS / 8;
    }
    static __host__ __device__ constexpr int64_t v_byte(int t, int dim) {
        return int64_t(t / 16) * 16 * kRow +
               (((t % 16 / 4 * 16 + dim % 16) * 2 + t % 4 / 2) * kUnits + dim / kUnitDims) * 4 + t % 2 * 2 +
               dim % kUnitDims / 16 * BITS / 8;
    }
    static __host__ __device__ constexpr int k_nibble(int dim) { return BITS == 4 ? dim % 2 : 0; }
    static __host__ __device__ constexpr int v_nibble(int dim) { return BITS == 4 ? dim / 16 % 2 : 0; }
};

inline int64_t kv_chunk_bytes(int bits, int64_t page_tokens, int64_t dim) {
    return 2 * page_tokens * (dim * bits / 8 + dim / 16);
}

// f(bits, dim) with the cache's kind as compile-time constants.
template <class F>
void kv_kinds(int bits, int64_t dim, const F& f) {
    auto dims = [&](auto b) {
        if (dim == 64) f(b, std::integral_constant<int, 64>{});
        else if (dim == 128) f(b, std::integral_constant<int, 128>{});
        else f(b, std::integral_constant<int, 256>{});
    };
    if (bits == 4) dims(std::integral_constant<int, 4>{});
    else dims(std::integral_constant<int, 8>{});
}

// The token's sequence and its position in that sequence's cache; seq < 0 for a row of no sequence.
// Every lane of the wave is active; starts and lengths are read together, 64 sequences at a time.
struct KvToken {
    int seq, pos;
};
__device__ __forceinline__ KvToken kv_token(const KvView& c, int t) {
    const int lane = threadIdx.x & 63;
    if (t < c.q_start[0]) return {-1, 0};
    for (int i0 = 0; i0 < c.seqs; i0 += 64) {
        const int i = min(i0 + lane, c.seqs - 1);
        const int end = c.q_start[i + 1], len = c.kv_len[i];
        const int past = __popcll(__ballot(end <= t));
        if (past < 64) {     // (starts do not fall: the first sequence that ends behind the token; lanes behind the last repeat it)
            const int b = __builtin_amdgcn_readfirstlane(past);
            if (i0 + b >= c.seqs) return {-1, 0};     // (starts that fall: no such sequence, and no read behind the table)
            const unsigned behind = unsigned(__builtin_amdgcn_readlane(end, b)) - unsigned(t);
            return {i0 + b, int(unsigned(__builtin_amdgcn_readlane(len, b)) - behind)};
        }
    }
    return {-1, 0};
}

// Page of position `pos` of sequence b, or -1 where the table has none (also a page outside the cache).
__device__ __forceinline__ int kv_page(const KvView& c, int b, int pos) {
    const int at = pos >> c.page_shift;
    if (pos < 0 || at >= c.width) return -1;
    const int p = c.table[int64_t(b) * c.width + at];
    return p >= 0 && p < c.pages ? p : -1;
}

}  // namespace mq
