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
    uint32_t per_head, per_page;  // kv_per(nheads), kv_per(page_size)
};

// Quotients of numbers up to 2^31 by n through 2^32 / n, rounded down and below 2^32: at most one too low.
inline uint32_t kv_per(int n) { return n == 1 ? ~0u : (uint32_t)((1ull << 32) / (unsigned)n); }
__device__ __forceinline__ uint32_t kv_divide(uint32_t v, uint32_t n, uint32_t per, uint32_t& rest) {
    uint32_t q = (uint32_t)(((uint64_t)v * per) >> 32);
    rest = v - q * n;
    if (rest >= n) {
        rest -= n;
        ++q;
    }
    return q;
}

__host__ __device__ constexpr int kv_factor_bytes(int type, int dim) { return type == kKvF16 ? 2 * dim : type == kKvQ8 ? dim : dim / 2; }
__host__ __device__ constexpr int kv_row_bytes(int type, int dim) { return kv_factor_bytes(type, dim) + (type == kKvF16 ? 0 : dim / 16); }

// 2^e for e in [-126, 127]
__device__ __forceinline__ float power(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

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

// The sequence of token t with the end of its new tokens and its length, or -1: one more than the sequences
// that end at or before it.  By the 16 lanes of a row (each with the same t): the sixteenths of what is left until
// it is 16 sequences, whose ends and lengths arrive together.
__device__ __forceinline__ int sum16(int v) {
    v += dpp_i<0xB1>(v);
    v += dpp_i<0x4E>(v);
    v += dpp_i<0x141>(v);
    v += dpp_i<0x140>(v);
    return v;
}
__device__ __forceinline__ int kv_sequence16(const KvPlace& p, int t, int& end, int& len) {
    end = t + 1;
    if (!p.seg_off) {
        len = t < p.nseq ? p.lens[t] : 0;
        return t < p.nseq ? t : -1;
    }
    const int i = threadIdx.x & 15;
    int from = 0, n = p.nseq;  // the sequence is one of the n from `from` on, or none
    while (n > 16) {
        const int step = (n + 15) / 16, last = (i + 1) * step;
        const int over = sum16(last < n && min(max(p.seg_off[from + last], 0), p.ntok) <= t ? 1 : 0) * step;
        from += over;
        n = min(step, n - over);
    }
    const int at_most = from + min(i, max(n, 1) - 1);  // (nseq > 0: all three arrive together)
    const int begin = p.seg_off[0], l = p.lens[min(at_most, p.nseq - 1)], e = min(max(p.seg_off[min(at_most, p.nseq - 1) + 1], 0), p.ntok);
    const int over = sum16(i < n && e <= t ? 1 : 0), at = 4 * ((threadIdx.x & 48) + min(over, 15));
    end = __builtin_amdgcn_ds_bpermute(at, e);
    len = __builtin_amdgcn_ds_bpermute(at, l);
    return over < n && begin <= t ? from + over : -1;
}

// The page of position pos of sequence s and the place there, or -1 (and a place) where there is none; s in
// [0, nseq).
__device__ __forceinline__ int kv_page(const KvPlace& p, int s, int64_t pos, int& place) {
    const bool in = pos >= 0 && pos < (int64_t)p.max_pages * p.page_size;
    uint32_t rest;
    const uint32_t at = kv_divide(in ? (uint32_t)pos : 0, p.page_size, p.per_page, rest);
    place = (int)rest;
    const int pg = p.pages[(int64_t)s * p.ldpages + at];
    return in && pg >= 0 && pg < p.npages ? pg : -1;
}

// The chunk of a page and head.
__device__ __forceinline__ char* kv_chunk(const KvSide& c, const KvPlace& p, int page, int head) {
    return c.base + page * c.stride + (int64_t)head * p.page_size * kv_row_bytes(c.type, p.dim);
}

}  // namespace qmm
