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
    int type, sides;
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

// Two values rounded to a type of 16 bits, to nearest even, in one instruction.
__device__ __forceinline__ uint32_t pair_of(int type, float v, float w) {
    typedef float float2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
    const float2_t both = {v, w};
    return type == kBin16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(both, half2_t))
                          : __builtin_bit_cast(uint32_t, __builtin_convertvector(both, bf2_t));
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

// Row of a 16-lane group: rows are (token, head); those past the last are the last, and not live.  Every lane of a
// wave goes the same way from here on.
struct KvRow {
    int t, h, n;  // n: the lane of the group
    bool live;
    __device__ __forceinline__ explicit KvRow(const KvPlace& p) {
        const uint32_t all = p.ntok * p.nheads, at = blockIdx.x * 16 + threadIdx.x / 16;
        uint32_t rest;
        t = (int)kv_divide(min(at, all - 1), p.nheads, p.per_head, rest);
        h = (int)rest;
        n = threadIdx.x & 15;
        live = at < all;
    }
};
// Its sequence, or -1; its position's page, or -1, and place there.
struct KvSpot {
    int seq, page, place;
    __device__ __forceinline__ KvSpot(const KvPlace& p, const KvRow& row) {
        int end, len;
        seq = kv_sequence16(p, row.t, end, len);
        page = kv_page(p, max(seq, 0), (int64_t)len - (end - row.t), place);
        if (seq < 0) page = -1;
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
//   8192 tokens of 4 heads of 128, binary16 to q8_0, keys and values: 12.6 us, 2.0 TB/s
// (17.7 with every quotient divided out and a byte a store); 8 tokens: 3.9 us, two dependent loads and a launch.
template <int NB>
struct KvWrite {
    uint32_t raw[2 * NB], table;
    __device__ __forceinline__ void load(const KvRows& a, int which, const KvRow& row) {
        const int64_t from = row.t * a.ld[which] + (int64_t)row.h * (32 * NB);
        if (a.side[which].type == kKvF16) {
            if (a.type == kF32) __builtin_memcpy(raw, (const float*)a.x[which] + from + 2 * NB * row.n, 8 * NB);
            else __builtin_memcpy(raw, (const uint16_t*)a.x[which] + from + 2 * NB * row.n, 4 * NB);
            return;
        }
        if (a.type == kF32) {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) raw[i] = ((const uint32_t*)a.x[which])[from + 16 * i + row.n];
        } else {
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) raw[i] = ((const uint16_t*)a.x[which])[from + 16 * i + row.n];
        }
        table = kIq4Table.word[threadIdx.x & 63];
    }
    __device__ __forceinline__ void store(const KvRows& a, int which, const KvRow& row, const KvSpot& spot) const {
        const int type = a.side[which].type, n = row.n;
        char* chunk = kv_chunk(a.side[which], a.p, max(spot.page, 0), row.h);
        const bool to_store = row.live && spot.page >= 0;
        if (type == kKvF16) {
            uint32_t w[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if (a.type == kF32) w[b] = pair_of(kBin16, __builtin_bit_cast(float, raw[2 * b]), __builtin_bit_cast(float, raw[2 * b + 1]));
                else if (a.type == kBf16) w[b] = pair_of(kBin16, bf2f(raw[b]), __builtin_bit_cast(float, raw[b] & 0xFFFF0000u));
                else w[b] = raw[b];
            }
            if (to_store) __builtin_memcpy(__builtin_assume_aligned(chunk + spot.place * (64 * NB) + 4 * NB * n, 4), w, 4 * NB);
            return;
        }
        float x[2 * NB];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) x[i] = a.type == kF32 ? __builtin_bit_cast(float, raw[i]) : a.type == kBin16 ? h2f(raw[i]) : bf2f(raw[i]);
        uint32_t scales[(NB + 1) / 2] = {}, out[(NB + 1) / 2] = {};
        const float* v = x;
        if (type == kKvQ8) {
#pragma unroll
            for (int b = 0; b < NB; ++b, v += 2) {
                const float amax = max16(__builtin_fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])));
                float d = over127(amax);
                const float per = __builtin_amdgcn_rcpf(d), r0 = __builtin_rintf(v[0] * per), r1 = __builtin_rintf(v[1] * per);
                int q0 = (int)r0, q1 = (int)r1;
                const bool sure = sure_scale(d) && __builtin_fabsf(v[0] * per - r0) <= 0.49995f && __builtin_fabsf(v[1] * per - r1) <= 0.49995f;
                if (__any(!sure)) {
                    d = amax / 127.0f;
                    q0 = d == 0.0f ? 0 : min(max(round_away(v[0] / d), -127), 127);
                    q1 = d == 0.0f ? 0 : min(max(round_away(v[1] / d), -127), 127);
                }
                out[b / 2] |= (uint32_t)((q0 & 255) | (q1 & 255) << 8) << (16 * (b & 1));
                scales[b / 2] |= f2h(d) << (16 * (b & 1));
            }
            if (to_store) __builtin_memcpy(chunk + (spot.place * 16 + n) * (2 * NB), out, 2 * NB);
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b, v += 2) {
                const float amax = max16(__builtin_fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])));
                // the first value of that magnitude: its index in the block, its sign in bit 0
                const int mine = __builtin_fabsf(v[0]) == amax ? 2 * n + (v[0] < 0.0f) : __builtin_fabsf(v[1]) == amax ? 2 * (n + 16) + (v[1] < 0.0f) : 64;
                const bool negative = min16(mine) & 1;
                float d = over127(amax);
                bool sure = sure_scale(d);
                d = negative ? d : -d;
                const float per = __builtin_amdgcn_rcpf(d);
                int q[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float u = v[i] * (2.0f * per);
                    // the lane: u / 8 + 32 in the eighths of [2^20, 2^21)
                    const uint32_t lane = __builtin_bit_cast(uint32_t, __builtin_fmaf(v[i], 0.25f * per, 1572864.0f + 32.0f));
                    const uint32_t word = (uint32_t)__builtin_amdgcn_ds_bpermute((int)(lane >> 1 & 252), (int)table);
                    const float middle = __builtin_bit_cast(float, word);
                    sure &= __builtin_fabsf(u - middle) >= power(-10);
                    q[i] = (int)(word & 15) + (u > middle ? 1 : 0);
                }
                if (__any(!sure)) {
                    d = (negative ? -amax : amax) / -127.0f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) q[i] = d == 0.0f ? 8 : iq4nl_nearest(v[i] / d);
                    d = d == 0.0f ? 0.0f : d;
                }
                out[b / 4] |= (uint32_t)(q[0] | q[1] << 4) << (8 * (b & 3));
                scales[b / 2] |= f2h(d) << (16 * (b & 1));
            }
            if (to_store) __builtin_memcpy(chunk + (spot.place * 16 + n) * NB, out, NB);
        }
        if (to_store && n == 0) __builtin_memcpy(chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB) + spot.place * (2 * NB), scales, 2 * NB);
    }
    static __device__ __forceinline__ float over127(float v) {
        constexpr float kPer = 1.0f / 127.0f;
        const float near = v * kPer;
        return __builtin_fmaf(__builtin_fmaf(-near, 127.0f, v), kPer, near);
    }
    static __device__ __forceinline__ bool sure_scale(float d) { return d >= power(-100) && d < power(120); }
};

template <int NB>
__global__ __launch_bounds__(256) void kv_write_kernel(KvRows a) {
    const KvRow row(a.p);
    KvWrite<NB> one;
    if (gridDim.y == 1 && a.sides == 2) {
        KvWrite<NB> two;
        one.load(a, 0, row);
        two.load(a, 1, row);
        const KvSpot spot(a.p, row);
        one.store(a, 0, row, spot);
        two.store(a, 1, row, spot);
    } else {
        one.load(a, blockIdx.y, row);
        one.store(a, blockIdx.y, row, KvSpot(a.p, row));
    }
}

// Two neighbouring values of a row.
__device__ __forceinline__ void store_pair(void* p, int64_t i, int type, float v, float w) {
    if (type == kF32) {
        const float both[2] = {v, w};
        __builtin_memcpy((float*)p + i, both, 8);
    } else {
        const uint32_t both = pair_of(type, v, w);
        __builtin_memcpy((uint16_t*)p + i, &both, 4);
    }
}

// As the writes; of a block format lanes n and n + 1 exchange a value of each block, and store two neighbours: 8192
// positions of 4 heads of 128, q8_0 to binary16, keys and values in 9.2 us, 2.8 TB/s (14.5 a value a store); bound by
// the instructions a value costs and by one load after the other.
template <int NB>
struct KvRead {
    uint32_t f[NB] = {}, scales[(NB + 1) / 2] = {};
    __device__ __forceinline__ void load(const KvRows& a, int which, const KvRow& row, const KvSpot& spot) {
        const int type = a.side[which].type, n = row.n;
        if (spot.page < 0) {
            // +0 of every format: a scale of zero times the level 1, where index 0 is -127
            if (type == kKvIq4)
#pragma unroll
                for (int i = 0; i < NB; ++i) f[i] = 0x88888888u;
            return;
        }
        const char* chunk = kv_chunk(a.side[which], a.p, spot.page, row.h);
        if (type == kKvF16) {
            __builtin_memcpy(f, __builtin_assume_aligned(chunk + spot.place * (64 * NB) + 4 * NB * n, 4), 4 * NB);
            return;
        }
        if (type == kKvQ8) __builtin_memcpy(f, chunk + (spot.place * 16 + n) * (2 * NB), 2 * NB);
        else __builtin_memcpy(f, chunk + (spot.place * 16 + n) * NB, NB);
        __builtin_memcpy(scales, chunk + a.p.page_size * kv_factor_bytes(type, 32 * NB) + spot.place * (2 * NB), 2 * NB);
    }
    __device__ __forceinline__ void store(const KvRows& a, int which, const KvRow& row, const KvSpot& spot) const {
        const int type = a.side[which].type, n = row.n;
        const int64_t to = row.t * a.ld[which] + (int64_t)row.h * (32 * NB);
        const bool to_store = row.live && spot.seq >= 0;
        if (type == kKvF16) {
            if (!to_store) return;
            if (a.type == kBin16) {
                __builtin_memcpy((uint16_t*)a.y[which] + to + 2 * NB * n, f, 4 * NB);
            } else if (a.type == kF32) {
                float v[2 * NB];
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) v[i] = h2f(f[i / 2] >> (16 * (i & 1)));
                __builtin_memcpy((float*)a.y[which] + to + 2 * NB * n, v, 8 * NB);
            } else {
                uint32_t w[NB];
#pragma unroll
                for (int b = 0; b < NB; ++b) w[b] = pair_of(kBf16, h2f(f[b]), h2f(f[b] >> 16));
                __builtin_memcpy((uint16_t*)a.y[which] + to + 2 * NB * n, w, 4 * NB);
            }
            return;
        }
        uint32_t lo[(NB + 3) / 4], hi[(NB + 3) / 4];
        if (type == kKvIq4) {
            const IQ4Levels levels;
#pragma unroll
            for (int i = 0; i < (NB + 3) / 4; ++i) iq4nl_decode_word(f[i], lo[i], hi[i], levels);
        } else {
            // the bytes of an even and an odd place apart
#pragma unroll
            for (int i = 0; i < (NB + 3) / 4; ++i) {
                const uint32_t next = 2 * i + 1 < (NB + 1) / 2 ? f[2 * i + 1] : 0;
                lo[i] = perm(next, f[2 * i], 0x06040200u);
                hi[i] = perm(next, f[2 * i], 0x07050301u);
            }
        }
        const bool odd = n & 1;
        float v[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float d = h2f(scales[b / 2] >> (16 * (b & 1)));
            const float v0 = opaque(d * (float)(int8_t)(lo[b / 4] >> (8 * (b & 3)))), v1 = opaque(d * (float)(int8_t)(hi[b / 4] >> (8 * (b & 3))));
            const float got = dpp<0xB1>(odd ? v0 : v1);
            v[b][0] = odd ? got : v0;
            v[b][1] = odd ? v1 : got;
        }
        if (!to_store) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) store_pair(a.y[which], to + 32 * b + (odd ? 15 : 0) + n, a.type, v[b][0], v[b][1]);
    }
};

template <int NB>
__global__ __launch_bounds__(256) void kv_read_kernel(KvRows a) {
    const KvRow row(a.p);
    const KvSpot spot(a.p, row);
    KvRead<NB> one;
    if (gridDim.y == 1 && a.sides == 2) {
        KvRead<NB> two;
        one.load(a, 0, row, spot);
        two.load(a, 1, row, spot);
        one.store(a, 0, row, spot);
        two.store(a, 1, row, spot);
    } else {
        one.load(a, blockIdx.y, row, spot);
        one.store(a, blockIdx.y, row, spot);
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
    // Both sides by the same workgroups, with one look-up, where they would otherwise not fit at once (8 on each of 256
    // CUs): 8192 tokens of 4 heads of 128 read in 9.3 us, apart in 10.1; 2048 tokens in 4.65, apart in 4.1.
    const int64_t groups = (ntok * c->nheads + 15) / 16;
    a.sides = n;
    launch(a, dim3((unsigned)groups, groups * n > 8 * 256 ? 1u : (unsigned)n));
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
