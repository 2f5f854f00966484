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
    uint32_t per_head;  // 2^32 / nheads, rounded down, below 2^32
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

// The same for u = 2v in [-254, 254], by the lanes of a wave: lane b of a table holds the one doubled middle in
// [8 (b - 32) - 1/2, 8 (b - 32) + 15/2), or a large number, and in its low four bits how many are below.
struct Iq4Table {
    uint32_t word[64];
    constexpr Iq4Table() : word() {
        const int mid[15] = {-231, -187, -148, -114, -84, -57, -32, -9, 14, 38, 63, 91, 122, 158, 202};
        for (int b = 0; b < 64; ++b) {
            const int low = 8 * (b - 32);
            int below = 0, in = 1 << 14;
            for (int i = 0; i < 15; ++i) {
                below += mid[i] < low ? 1 : 0;
                if (mid[i] >= low && mid[i] < low + 8) in = mid[i];
            }
            word[b] = __builtin_bit_cast(uint32_t, (float)in) | (uint32_t)below;
        }
    }
};
__constant__ constexpr Iq4Table kIq4Table;

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

// Row of a 16-lane group: rows are (token, head), blockIdx.y the keys or the values.  Rows past the last are the
// last, and not live.  Every lane of a wave goes the same way from here on.
struct KvRow {
    int t, h;
    bool live;
    __device__ __forceinline__ explicit KvRow(const KvRows& a) {
        const uint32_t heads = a.p.nheads, all = a.p.ntok * heads, at = blockIdx.x * 16 + threadIdx.x / 16, row = min(at, all - 1);
        uint32_t q = (uint32_t)(((uint64_t)row * a.per_head) >> 32);  // at most one too low
        q += row - q * heads >= heads ? 1 : 0;
        t = (int)q;
        h = (int)(row - q * heads);
        live = at < all;
    }
    // Its sequence, or -1; its position's chunk (null: none) and place there.
    __device__ __forceinline__ int find(const KvRows& a, char*& chunk, int& place) const {
        int end, len, pg = -1;
        const int s = kv_sequence16(a.p, t, end, len);
        const int64_t pos = (int64_t)len - (end - t);
        if (s >= 0) pg = kv_page(a.p, s, pos);
        chunk = pg < 0 ? nullptr : kv_chunk(a.side[blockIdx.y], a.p, pg, h);
        place = pg < 0 ? 0 : (int)((uint32_t)pos % (uint32_t)a.p.page_size);
        return s;
    }
};

// Sixteen lanes a row; lane n holds values n and n + 16 of every block, which are the contiguous bytes of a
// block format's row that it writes, and a block's maximum is a maximum over the lanes; of binary16 a sixteenth
// of the row.  The row is read before its place is looked up: a few tokens cost the longer of the two chains of
// loads.
//   Many tokens are bound by the instructions a value costs, so quotients are not divided out: amax / 127 is its
// product with 1 / 127 and one residual step (the correctly rounded quotient for each of the 2^23 significands,
// checked one by one), x / d the product with a reciprocal.  That is within 2^-22 of it, and its rounding certain unless it
// lies within 5e-5 of a tie (2^-10 of a doubled middle): then, and for a scale beyond what this holds for,
// zero or not finite, or a NaN, the wave divides the block again as the definition does.
template <int NB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRows a) {
    const KvRow row(a);
    const int which = blockIdx.y, n = threadIdx.x & 15, type = a.side[which].type;
    const int64_t from = row.t * a.ld[which] + (int64_t)row.h * (32 * NB);
    char* chunk;
    int place;
    if (type == kKvF16) {
        uint32_t raw[2 * NB], w[NB];
        if (a.type == kF32) __builtin_memcpy(raw, (const float*)a.x[which] + from + 2 * NB * n, 8 * NB);
        else __builtin_memcpy(raw, (const uint16_t*)a.x[which] + from + 2 * NB * n, 4 * NB);
        row.find(a, chunk, place);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (a.type == kF32) w[b] = f2h(__builtin_bit_cast(float, raw[2 * b])) | f2h(__builtin_bit_cast(float, raw[2 * b + 1])) << 16;
            else if (a.type == kBf16) w[b] = f2h(bf2f(raw[b])) | f2h(__builtin_bit_cast(float, raw[b] & 0xFFFF0000u)) << 16;
            else w[b] = raw[b];
        }
        if (row.live && chunk) __builtin_memcpy(__builtin_assume_aligned(chunk + place * (64 * NB) + 4 * NB * n, 4), w, 4 * NB);
        return;
    }
    uint32_t raw[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = from + 32 * b + 16 * i + n;
            raw[b][i] = a.type == kF32 ? ((const uint32_t*)a.x[which])[at] : ((const uint16_t*)a.x[which])[at];
        }
    const uint32_t table = type == kKvIq4 ? kIq4Table.word[threadIdx.x & 63] : 0;
    row.find(a, chunk, place);
    float x[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[b][i] = a.type == kF32 ? __builtin_bit_cast(float, raw[b][i]) : a.type == kBin16 ? h2f(raw[b][i]) : bf2f(raw[b][i]);
    uint32_t scales[(NB + 1) / 2] = {}, out[(NB + 1) / 2] = {};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const float amax = max16(__builtin_fmaxf(__builtin_fabsf(x[b][0]), __builtin_fabsf(x[b][1])));
        constexpr float kPer = 1.0f / 127.0f;
        const float near = amax * kPer;
        float d = __builtin_fmaf(__builtin_fmaf(-near, 127.0f, amax), kPer, near);
        bool again = !(d >= power(-100) && d < power(120));
        int q[2];
        if (type == kKvQ8) {
            const float per = __builtin_amdgcn_rcpf(d);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float v = x[b][i] * per, r = __builtin_rintf(v);
                again |= !(__builtin_fabsf(v - r) <= 0.49995f);
                q[i] = (int)r;
            }
            if (__any(again)) {
                d = amax / 127.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = round_away(x[b][i] / d);
                    q[i] = d == 0.0f ? 0 : r > 127 ? 127 : r < -127 ? -127 : r;
                }
            }
            out[b / 2] |= (uint32_t)((q[0] & 255) | (q[1] & 255) << 8) << (16 * (b & 1));
        } else {
            // the first value of that magnitude: its index in the block, its sign in bit 0
            const int mine = __builtin_fabsf(x[b][0]) == amax ? 2 * n + (x[b][0] < 0.0f)
                             : __builtin_fabsf(x[b][1]) == amax ? 2 * (n + 16) + (x[b][1] < 0.0f) : 64;
            const bool negative = min16(mine) & 1;
            d = negative ? d : -d;
            const float per = __builtin_amdgcn_rcpf(d);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float u = x[b][i] * (2.0f * per);
                // the lane: u / 8 + 32 in the eighths of [2^20, 2^21)
                const uint32_t lane = __builtin_bit_cast(uint32_t, __builtin_fmaf(x[b][i], 0.25f * per, 1572864.0f + 32.0f));
                const uint32_t word = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(lane >> 1 & 252), (int)table);
                const float middle = __builtin_bit_cast(float, word);
                again |= !(__builtin_fabsf(u - middle) >= power(-10));
                q[i] = (int)(word & 15) + (u > middle ? 1 : 0);
            }
            if (__any(again)) {
                d = (negative ? -amax : amax) / -127.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) q[i] = d == 0.0f ? 8 : iq4nl_nearest(x[b][i] / d);
                d = d == 0.0f ? 0.0f : d;
            }
            out[b / 4] |= (uint32_t)(q[0] | q[1] << 4) << (8 * (b & 3));
        }
        scales[b / 2] |= f2h(d) << (16 * (b & 1));
    }
    if (!row.live || !chunk) return;
    if (type == kKvQ8) __builtin_memcpy(chunk + (place * 16 + n) * (2 * NB), out, 2 * NB);
    else __builtin_memcpy(chunk + (place * 16 + n) * NB, out, NB);
    if (n == 0) __builtin_memcpy(chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB) + place * (2 * NB), scales, 2 * NB);
}

// Two neighbouring values of a row, each rounded to the output's type.
__device__ __forceinline__ void store_pair(void* p, int64_t i, int type, float v, float w) {
    if (type == kF32) {
        const float both[2] = {v, w};
        __builtin_memcpy((float*)p + i, both, 8);
    } else {
        const uint32_t both = type == kBin16 ? f2h(v) | f2h(w) << 16 : f2bf(v) | f2bf(w) << 16;
        __builtin_memcpy((uint16_t*)p + i, &both, 4);
    }
}

// As the writes; of a block format lanes n and n + 1 exchange a value of each block, and store two neighbours.
template <int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRows a) {
    const KvRow row(a);
    const int which = blockIdx.y, n = threadIdx.x & 15, type = a.side[which].type;
    const int64_t to = row.t * a.ld[which] + (int64_t)row.h * (32 * NB);
    char* chunk;
    int place;
    const int s = row.find(a, chunk, place);
    if (type == kKvF16) {
        uint32_t w[NB] = {};
        if (chunk) __builtin_memcpy(w, __builtin_assume_aligned(chunk + place * (64 * NB) + 4 * NB * n, 4), 4 * NB);
        if (!row.live || s < 0) return;
        if (a.type == kBin16) {
            __builtin_memcpy((uint16_t*)a.y[which] + to + 2 * NB * n, w, 4 * NB);
        } else {
            uint32_t v[2 * NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float lo = h2f(w[b]), hi = h2f(w[b] >> 16);
                v[2 * b] = a.type == kF32 ? __builtin_bit_cast(uint32_t, lo) : f2bf(lo) | f2bf(hi) << 16;
                v[2 * b + 1] = __builtin_bit_cast(uint32_t, hi);
            }
            if (a.type == kF32) {
                __builtin_memcpy((float*)a.y[which] + to + 2 * NB * n, v, 8 * NB);
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b) w[b] = v[2 * b];
                __builtin_memcpy((uint16_t*)a.y[which] + to + 2 * NB * n, w, 4 * NB);
            }
        }
        return;
    }
    uint32_t f[(NB + 1) / 2] = {}, scales[(NB + 1) / 2] = {}, lo[(NB + 3) / 4], hi[(NB + 3) / 4];
    if (chunk) {
        if (type == kKvQ8) __builtin_memcpy(f, chunk + (place * 16 + n) * (2 * NB), 2 * NB);
        else __builtin_memcpy(f, chunk + (place * 16 + n) * NB, NB);
        __builtin_memcpy(scales, chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB) + place * (2 * NB), 2 * NB);
    }
    if (type == kKvIq4) {
        const IQ4Levels levels;
#pragma unroll
        for (int i = 0; i < (NB + 3) / 4; ++i) iq4nl_decode_word(f[i], lo[i], hi[i], levels);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t q0 = type == kKvQ8 ? f[b / 2] >> (16 * (b & 1)) : lo[b / 4] >> (8 * (b & 3));
        const uint32_t q1 = type == kKvQ8 ? f[b / 2] >> (16 * (b & 1) + 8) : hi[b / 4] >> (8 * (b & 3));
        const float d = h2f(scales[b / 2] >> (16 * (b & 1)));
        const float v0 = opaque(d * (float)(int8_t)q0), v1 = opaque(d * (float)(int8_t)q1);
        const bool odd = n & 1;
        const float got = dpp<0xB1>(odd ? v0 : v1);
        if (row.live && s >= 0) store_pair(a.y[which], to + 32 * b + (odd ? 15 : 0) + n, a.type, odd ? got : v0, odd ? v1 : got);
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
    a.per_head = c->nheads == 1 ? ~0u : (uint32_t)((1ull << 32) / (unsigned)c->nheads);
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
