// qmm_attend.hip -- attention of new tokens over the paged key-value cache, for gfx950.
//
// For a row (token, head) at position p: z_j = scale q . k_j over the positions j it sees, out = sum_j
// exp(z_j - m) v_j / sum_j exp(z_j - m) with the running maximum m and sum of one pass over the cache.
#include "qmm_kv.h"

namespace qmm {

struct AttendArgs {
    const void* q;
    void* out;
    float* lse;
    int64_t ldq, ldo;
    KvSide k, v;
    KvPlace p;
    int nheads, qtype, otype;
    float scale;
    int64_t window;
};

__device__ __forceinline__ float kv_value(const char* chunk, int type, int place, int dim, int page_size, int c) {
    if (type == kKvF16) return h2f(((const uint16_t*)chunk)[place * dim + c]);
    const int nb = dim / 32, b = c / 32, i = c / 16 & 1, n = c & 15;
    const float d = h2f(((const uint16_t*)(chunk + page_size * kv_factor_bytes(type, dim)))[place * nb + b]);
    if (type == kKvQ8) return d * (float)((const int8_t*)chunk)[((place * 16 + n) * nb + b) * 2 + i];
    return d * iq4nl_value(((const uint8_t*)chunk)[(place * 16 + n) * nb + b] >> (4 * i) & 15);
}

// One wave per row: 64 positions at a time, a lane a score, then a lane every 64th value of the output.
__global__ __launch_bounds__(64) void attend_kernel(AttendArgs a) {
    __shared__ float q[256], w[64];
    __shared__ int at[64];
    const int t = (int)(blockIdx.x / (uint32_t)a.nheads), h = (int)(blockIdx.x - (uint32_t)t * a.nheads), lane = threadIdx.x;
    const int s = kv_sequence16(a.p, t);
    if (s < 0) return;
    const int dim = a.p.dim, head = h / (a.nheads / a.p.nheads), ps = a.p.page_size;
    int first, end;
    kv_segment(a.p, s, first, end);
    const int64_t pos = (int64_t)a.p.lens[s] - (end - t);
    for (int c = lane; c < dim; c += 64) q[c] = load_value(a.q, t * a.ldq + (int64_t)h * dim + c, a.qtype) * a.scale;
    __syncthreads();
    const int64_t hi = min(pos + 1, (int64_t)a.p.max_pages * ps);
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t j0 = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0; j0 < hi; j0 += 64) {
        const int64_t j = j0 + lane;
        const int pg = j < hi ? kv_page(a.p, s, j) : -1, place = (int)((uint32_t)j % (uint32_t)ps);
        float z = -INFINITY;
        if (pg >= 0) {
            const char* chunk = kv_chunk(a.k, a.p, pg, head);
            z = 0.0f;
            for (int c = 0; c < dim; ++c) z += q[c] * kv_value(chunk, a.k.type, place, dim, ps, c);
        }
        float top = z;
        for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i, 64));
        const float now = fmaxf(m, top), base = now == -INFINITY ? 0.0f : now;
        const float e = pg >= 0 ? expf(z - base) : 0.0f, shrink = expf(m - base);
        float total = e;
        for (int i = 1; i < 64; i <<= 1) total += __shfl_xor(total, i, 64);
        l = l * shrink + total;
        m = now;
        w[lane] = e;
        at[lane] = pg;
        __syncthreads();
        for (int i = 0; i < 4; ++i) {
            const int c = lane + 64 * i;
            o[i] *= shrink;
            if (c >= dim) continue;
            for (int x = 0; x < 64; ++x)
                if (at[x] >= 0)
                    o[i] += w[x] * kv_value(kv_chunk(a.v, a.p, at[x], head), a.v.type, (int)((uint32_t)(j0 + x) % (uint32_t)ps), dim, ps, c);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int c = lane + 64 * i;
        if (c < dim) store_value(a.out, t * a.ldo + (int64_t)h * dim + c, a.otype, l != 0.0f ? o[i] / l : 0.0f);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.nheads + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace qmm

#include "qmm_kv_host.h"

using namespace qmm;

static int attend_place(KvPlace& p, const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages,
                        const int32_t* lens, const int32_t* seg_off, int nseq, int64_t ntok, int nheads) {
    const int rc = kv_place(p, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok);
    if (rc != QMM_OK) return rc;
    if (nheads < 1 || nheads % c->nheads) return QMM_EINVAL;
    if (nheads > 1024 || ntok * nheads > kKvMaxRows || kv_row_bytes(c->vtype, 64) > kv_row_bytes(c->ktype, 64)) return QMM_EUNSUPPORTED;
    return QMM_OK;
}

extern "C" size_t qmm_kv_attend_workspace(const qmm_kv_cache* c, int64_t ntok, int nheads, int nseq, int64_t max_pages) {
    KvPlace p;
    static const int32_t some = 0;
    return attend_place(p, c, &some, max_pages, max_pages, &some, &some, nseq, ntok, nheads) == QMM_OK ? 16 : 0;
}

extern "C" int qmm_kv_attend(const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                             const int32_t* seg_off, int nseq, int qtype, const void* q, int64_t ldq, int64_t ntok, int nheads,
                             float scale, int64_t window, int otype, void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                             void* stream) {
    AttendArgs a;
    if (!valid_type(qtype) || !valid_type(otype) || window < 0 || !(scale >= -3.4e38f) || !(scale <= 3.4e38f)) return QMM_EINVAL;
    const int rc = attend_place(a.p, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok, nheads);
    if (rc != QMM_OK) return rc;
    const int64_t width = (int64_t)nheads * c->head_dim;
    if (ldq < width || ldo < width) return QMM_EINVAL;
    if (ntok == 0 || nseq == 0) return QMM_OK;
    if (!q || !out || !ws) return QMM_EINVAL;
    if (!aligned(q, type_bytes(qtype)) || !aligned(out, type_bytes(otype)) || !aligned(lse, 4) || !aligned(ws, 16)) return QMM_EALIGN;
    if (ws_bytes < qmm_kv_attend_workspace(c, ntok, nheads, nseq, max_pages)) return QMM_ESPACE;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.ldq = ldq;
    a.ldo = ldo;
    a.k = KvSide{(char*)c->k, c->kstride, c->ktype};
    a.v = KvSide{(char*)c->v, c->vstride, c->vtype};
    a.nheads = nheads;
    a.qtype = qtype;
    a.otype = otype;
    a.scale = scale;
    a.window = window;
    hipLaunchKernelGGL(attend_kernel, dim3((unsigned)(ntok * nheads)), dim3(64), 0, as_stream(stream), a);
    return launch_status();
}
