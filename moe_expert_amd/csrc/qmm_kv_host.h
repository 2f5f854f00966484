// qmm_kv_host.h -- argument checks of the entry points that take a qmm_kv_cache.  Host only.
#pragma once

#include "qmm_kv.h"
#include "qmm_types.h"

namespace qmm {

constexpr int64_t kKvMaxTokens = 1 << 20;
constexpr int kKvMaxSeq = 1 << 14;
constexpr int64_t kKvMaxLength = 0x40000000;  // positions of a sequence
constexpr int64_t kKvMaxRows = 1 << 27;  // 16 lanes a row, below 2^32 threads

inline bool kv_dim(int d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }
inline bool kv_type(int t) { return t == QMM_F16 || t == QMM_Q8_0 || t == QMM_IQ4_NL; }

// The cache by itself.
inline int kv_check(const qmm_kv_cache* c) {
    if (!c || !kv_type(c->ktype) || !kv_type(c->vtype) || c->npages < 1 || c->page_size < 1 || c->nheads < 1 || c->head_dim < 1)
        return QMM_EINVAL;
    if (!kv_dim(c->head_dim) || c->page_size % 16 || c->page_size > 4096 || c->nheads > 1024 || c->npages > 0x7FFFFFFF)
        return QMM_EUNSUPPORTED;
    const int64_t rows = (int64_t)c->nheads * c->page_size;
    if (c->kstride < rows * kv_row_bytes(c->ktype, c->head_dim) || c->vstride < rows * kv_row_bytes(c->vtype, c->head_dim))
        return QMM_EINVAL;
    if (!c->k || !c->v) return QMM_EINVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->kstride % 16 || c->vstride % 16) return QMM_EALIGN;
    return QMM_OK;
}

// The cache and a call's sequences.
inline int kv_place(KvPlace& p, const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                    const int32_t* seg_off, int nseq, int64_t ntok) {
    const int rc = kv_check(c);
    if (rc != QMM_OK) return rc;
    if (ntok < 0 || nseq < 0 || max_pages < 1 || ldpages < max_pages || (!seg_off && nseq != ntok)) return QMM_EINVAL;
    if (ntok > kKvMaxTokens || nseq > kKvMaxSeq || max_pages > kKvMaxLength || max_pages * c->page_size > kKvMaxLength) return QMM_EUNSUPPORTED;
    if (ntok && nseq && (!pages || !lens)) return QMM_EINVAL;
    if (!aligned(pages, 4) || !aligned(lens, 4) || !aligned(seg_off, 4)) return QMM_EALIGN;
    p = KvPlace{pages, lens, seg_off, ldpages, c->npages, (int)max_pages, c->page_size, c->nheads, c->head_dim, nseq, (int)ntok,
                kv_per(c->nheads), kv_per(c->page_size)};
    return QMM_OK;
}

}  // namespace qmm
