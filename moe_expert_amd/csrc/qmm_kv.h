// qmm_kv.h -- the paged key-value cache as the kernels see it: where a token's position lies, and the
// places of a block format's values.
#pragma once

#include "qmm_values.h"

namespace qmm {

enum : int { kKvQ8 = 1, kKvIq4 = 2, kKvF16 = 4 };  // QMM_Q8_0, QMM_IQ4_NL, QMM_F16

// One of the two arrays of a cache.
struct KvSide {
    char* base;
    int64_t stride;  // bytes from a page to the next
    int type;
};

struct KvPlace {
    const int32_t *pages, *lens, *seg_off;
    int64_t ldpages;
    int64_t npages;
    int max_pages, page_size, nheads, dim, nseq, ntok;
};

__host__ __device__ constexpr int kv_factor_bytes(int type, int dim) { return type == kKvF16 ? 2 * dim : type == kKvQ8 ? dim : dim / 2; }
__host__ __device__ constexpr int kv_row_bytes(int type, int dim) { return kv_factor_bytes(type, dim) + (type == kKvF16 ? 0 : dim / 16); }

__device__ __forceinline__ float iq4nl_value(int i) {
    return (float)(int8_t)((i & 8 ? 0x7159453526190D01ull : 0xF6EADDCFBFAD9881ull) >> (8 * (i & 7)));
}

// The first and last + 1 token of sequence s.
__device__ __forceinline__ void kv_segment(const KvPlace& p, int s, int& first, int& end) {
    if (!p.seg_off) {
        first = s;
        end = s + 1;
        return;
    }
    first = min(max(p.seg_off[s], 0), p.ntok);
    end = min(max(p.seg_off[s + 1], first), p.ntok);
}

// The sequence of token t, or -1: how many sequences end at or before it, counted by the 16 lanes of a
// row (each with the same t).
__device__ __forceinline__ int kv_sequence16(const KvPlace& p, int t) {
    if (!p.seg_off) return t < p.nseq ? t : -1;
    int n = 0;
    for (int i = threadIdx.x & 15; i < p.nseq; i += 16) n += min(max(p.seg_off[i + 1], 0), p.ntok) <= t ? 1 : 0;
    n += dpp_i<0xB1>(n);
    n += dpp_i<0x4E>(n);
    n += dpp_i<0x141>(n);
    n += dpp_i<0x140>(n);
    return n < p.nseq && max(p.seg_off[n], 0) <= t ? n : -1;
}

// The page of position pos of sequence s, or -1 where there is none.
__device__ __forceinline__ int kv_page(const KvPlace& p, int s, int64_t pos) {
    if (pos < 0 || pos >= (int64_t)p.max_pages * p.page_size) return -1;
    const int pg = p.pages[(int64_t)s * p.ldpages + (uint32_t)pos / (uint32_t)p.page_size];
    return pg >= 0 && pg < p.npages ? pg : -1;
}

// The chunk of a page and head.
__device__ __forceinline__ char* kv_chunk(const KvSide& c, const KvPlace& p, int page, int head) {
    return c.base + page * c.stride + (int64_t)head * p.page_size * kv_row_bytes(c.type, p.dim);
}

}  // namespace qmm
