// qmm_kv.hip -- the paged key-value cache: new tokens written, quantized per 32 values, and positions read
// back, for gfx950.
#include "qmm_kv.h"

namespace qmm {

struct KvRows {
    const void* x[2];
    void* y[2];
    int64_t ld[2];
    KvSide side[2];
    KvPlace p;
    int type;
};

// The index of the level nearest to v, ties to the lower one: the levels whose upper neighbour's middle v
// passes.  The middles are exact in binary32.
__device__ __forceinline__ int iq4nl_nearest(float v) {
    constexpr float mid[15] = {-115.5f, -93.5f, -74.0f, -57.0f, -42.0f, -28.5f, -16.0f, -4.5f,
                               7.0f,    19.0f,  31.5f,  45.5f,  61.0f,  79.0f,  101.0f};
    int n = 0;
#pragma unroll
    for (int i = 0; i < 15; ++i) n += v > mid[i] ? 1 : 0;
    return n;
}

__device__ __forceinline__ float max16(float v) {
    v = __builtin_fmaxf(v, dpp<0xB1>(v));
    v = __builtin_fmaxf(v, dpp<0x4E>(v));
    v = __builtin_fmaxf(v, dpp<0x141>(v));
    v = __builtin_fmaxf(v, dpp<0x140>(v));
    return v;
}
__device__ __forceinline__ int min16(int v) {
    v = min(v, dpp_i<0xB1>(v));
    v = min(v, dpp_i<0x4E>(v));
    v = min(v, dpp_i<0x141>(v));
    v = min(v, dpp_i<0x140>(v));
    return v;
}

// Row and cache of a 16-lane group: rows are (token, head), blockIdx.y the keys or the values.
__device__ __forceinline__ bool kv_row(const KvRows& a, int& t, int& h, char*& chunk, int& place) {
    const uint32_t row = blockIdx.x * 16 + threadIdx.x / 16;
    t = (int)(row / (uint32_t)a.p.nheads);
    h = (int)(row - (uint32_t)t * a.p.nheads);
    if (t >= a.p.ntok) return false;
    const int s = kv_sequence16(a.p, t);
    if (s < 0) return false;
    int first, end;
    kv_segment(a.p, s, first, end);
    const int64_t pos = (int64_t)a.p.lens[s] - (end - t);
    const int pg = kv_page(a.p, s, pos);
    chunk = pg < 0 ? nullptr : kv_chunk(a.side[blockIdx.y], a.p, pg, h);
    place = pg < 0 ? 0 : (int)((uint32_t)pos % (uint32_t)a.p.page_size);
    return true;
}

// Sixteen lanes a row; lane n holds values n and n + 16 of every block, which are the contiguous bytes of a
// block format's row that it writes, and a block's maximum is a maximum over the lanes.
template <int NB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRows a) {
    int t, h, place;
    char* chunk;
    if (!kv_row(a, t, h, chunk, place) || !chunk) return;
    const int which = blockIdx.y, n = threadIdx.x & 15, type = a.side[which].type;
    const int64_t at = t * a.ld[which] + (int64_t)h * (32 * NB);
    float x[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        for (int i = 0; i < 2; ++i) x[b][i] = load_value(a.x[which], at + 32 * b + 16 * i + n, a.type);
    if (type == kKvF16) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
            for (int i = 0; i < 2; ++i) ((uint16_t*)chunk)[place * (32 * NB) + 32 * b + 16 * i + n] = (uint16_t)f2h(x[b][i]);
        return;
    }
    uint16_t* scales = (uint16_t*)(chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB)) + place * NB;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const float amax = max16(__builtin_fmaxf(__builtin_fabsf(x[b][0]), __builtin_fabsf(x[b][1])));
        if (type == kKvQ8) {
            const float d = amax / 127.0f;
            int q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = round_away(x[b][i] / d);
                q[i] = d == 0.0f ? 0 : r > 127 ? 127 : r < -127 ? -127 : r;
            }
            ((uint16_t*)chunk)[(place * 16 + n) * NB + b] = (uint16_t)((q[0] & 255) | (q[1] & 255) << 8);
            if (n == 0) scales[b] = (uint16_t)f2h(d);
        } else {
            // the first value of that magnitude: its index in the block, its sign in bit 0
            const int mine = __builtin_fabsf(x[b][0]) == amax ? 2 * n + (x[b][0] < 0.0f)
                             : __builtin_fabsf(x[b][1]) == amax ? 2 * (n + 16) + (x[b][1] < 0.0f) : 64;
            const float d = (min16(mine) & 1 ? -amax : amax) / -127.0f;
            int q[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) q[i] = d == 0.0f ? 8 : iq4nl_nearest(x[b][i] / d);
            ((uint8_t*)chunk)[(place * 16 + n) * NB + b] = (uint8_t)(q[0] | q[1] << 4);
            if (n == 0) scales[b] = d == 0.0f ? 0 : (uint16_t)f2h(d);
        }
    }
}

template <int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRows a) {
    int t, h, place;
    char* chunk;
    if (!kv_row(a, t, h, chunk, place)) return;
    const int which = blockIdx.y, n = threadIdx.x & 15, type = a.side[which].type;
    const int64_t at = t * a.ld[which] + (int64_t)h * (32 * NB);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float v[2] = {0.0f, 0.0f};
        if (chunk) {
            const uint16_t* scales = (const uint16_t*)(chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB)) + place * NB;
            if (type == kKvF16) {
                for (int i = 0; i < 2; ++i) v[i] = h2f(((const uint16_t*)chunk)[place * (32 * NB) + 32 * b + 16 * i + n]);
            } else if (type == kKvQ8) {
                const uint32_t q = ((const uint16_t*)chunk)[(place * 16 + n) * NB + b];
                const float d = h2f(scales[b]);
                v[0] = opaque(d * (float)(int8_t)q);
                v[1] = opaque(d * (float)(int8_t)(q >> 8));
            } else {
                const int q = ((const uint8_t*)chunk)[(place * 16 + n) * NB + b];
                const float d = h2f(scales[b]);
                v[0] = opaque(d * iq4nl_value(q & 15));
                v[1] = opaque(d * iq4nl_value(q >> 4));
            }
        }
        for (int i = 0; i < 2; ++i) store_value(a.y[which], at + 32 * b + 16 * i + n, a.type, v[i]);
    }
}

}  // namespace qmm

#include "qmm_kv_host.h"

using namespace qmm;

// One launch over rows of 16 lanes; `only` is the side whose pointer is not null, or -1 for both.
template <class F>
static int kv_rows(const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                   const int32_t* seg_off, int nseq, int type, const void* k, int64_t ldk, const void* v, int64_t ldv,
                   int64_t ntok, F launch) {
    if (!valid_type(type) || (!k && !v && ntok != 0)) return QMM_EINVAL;
    KvRows a;
    int rc = kv_place(a.p, c, pages, ldpages, max_pages, lens, seg_off, nseq, ntok);
    if (rc != QMM_OK) return rc;
    const int64_t width = (int64_t)c->nheads * c->head_dim;
    if ((k && ldk < width) || (v && ldv < width)) return QMM_EINVAL;
    if (ntok * c->nheads > kKvMaxRows) return QMM_EUNSUPPORTED;
    if (ntok == 0 || nseq == 0) return QMM_OK;
    if ((k && !aligned(k, type_bytes(type))) || (v && !aligned(v, type_bytes(type)))) return QMM_EALIGN;
    a.type = type;
    const KvSide sides[2] = {{(char*)c->k, c->kstride, c->ktype}, {(char*)c->v, c->vstride, c->vtype}};
    const void* x[2] = {k, v};
    const int64_t ld[2] = {ldk, ldv};
    int n = 0;
    for (int i = 0; i < 2; ++i) {
        if (!x[i]) continue;
        a.x[n] = x[i];
        a.y[n] = const_cast<void*>(x[i]);
        a.ld[n] = ld[i];
        a.side[n++] = sides[i];
    }
    launch(a, dim3((unsigned)((ntok * c->nheads + 15) / 16), (unsigned)n));
    return launch_status();
}

#define QMM_BY_BLOCKS(kernel, dim, ...)                                        \
    switch ((dim) / 32) {                                                      \
        case 2: hipLaunchKernelGGL(kernel<2>, __VA_ARGS__); break;             \
        case 3: hipLaunchKernelGGL(kernel<3>, __VA_ARGS__); break;             \
        case 4: hipLaunchKernelGGL(kernel<4>, __VA_ARGS__); break;             \
        case 6: hipLaunchKernelGGL(kernel<6>, __VA_ARGS__); break;             \
        default: hipLaunchKernelGGL(kernel<8>, __VA_ARGS__); break;            \
    }

extern "C" int qmm_kv_write(const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                            const int32_t* seg_off, int nseq, int xtype, const void* k, int64_t ldk, const void* v, int64_t ldv,
                            int64_t ntok, void* stream) {
    return kv_rows(c, pages, ldpages, max_pages, lens, seg_off, nseq, xtype, k, ldk, v, ldv, ntok, [&](const KvRows& a, dim3 grid) {
        QMM_BY_BLOCKS(kv_write_kernel, c->head_dim, grid, dim3(256), 0, as_stream(stream), a)
    });
}

extern "C" int qmm_kv_read(const qmm_kv_cache* c, const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                           const int32_t* seg_off, int nseq, int otype, void* k, int64_t ldk, void* v, int64_t ldv, int64_t ntok,
                           void* stream) {
    return kv_rows(c, pages, ldpages, max_pages, lens, seg_off, nseq, otype, k, ldk, v, ldv, ntok, [&](const KvRows& a, dim3 grid) {
        QMM_BY_BLOCKS(kv_read_kernel, c->head_dim, grid, dim3(256), 0, as_stream(stream), a)
    });
}
