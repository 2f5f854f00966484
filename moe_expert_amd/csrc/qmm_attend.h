// qmm_attend.h -- the attention kernels over the paged key-value cache, for gfx950: one pass over the keys and
// values with the running maximum and sum of a softmax, split over the cache's length, and the join of the parts.
//
// For a row (token, head) at position p: z_j = scale q . k_j over the positions j it sees, out = sum_j
// exp(z_j - m) v_j / sum_j exp(z_j - m).
//
// A wave takes 32 positions a step against 16 rows of queries that share a head of keys (RT = 2: 32 rows).
// Scores come transposed, S^T = K Q^T by v_mfma_f32_16x16x32_f16: lane (n = l % 16, g = l / 16) gets, of row n,
// the positions 4g .. 4g+3 of both 16-position halves.  That is the operand of O^T = V^T P^T as it stands when
// the contraction runs over positions in the order (g, half, 0..3), so no weight moves between lanes, and every
// statistic of a row belongs to its lane.
//
// Nothing is rounded on the way that binary32 would keep: a block's integers are exact in binary16 (as
// (u - 128) 2^-10 of the biased byte u), its scale joins behind the products of the keys (one instruction a
// score and block) and before those of the values, into the weights; queries and weights enter in two
// binary16 parts, 2^-22 of the value in all, after a power of two a row that puts the largest near 2^14, so the second
// part keeps 2^-24 2^-14 of it.  One part alone would cost 2^-11, the error of a binary16 output.
#pragma once

#include "qmm_kv.h"

namespace qmm {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));
typedef float float4_t __attribute__((ext_vector_type(4)));

constexpr int kAtWaves = 4;      // waves of a workgroup, which take turns at the steps of a part
constexpr int kAtStep = 32;      // positions a step
constexpr int kAtInline = 256;   // sequences that a workgroup plans by itself; beyond, a launch of its own

struct AttendArgs {
    const void* q;
    void* out;
    float* lse;
    float* parts;            // partial results: [slot][head][rows (m), rows (l), rows * dim]
    const int32_t* plan;     // of attend_plan_kernel, or null
    int64_t ldq, ldo;
    KvSide k, v;
    KvPlace p;
    int nheads, group, qtype, otype;  // group: heads of queries a head of keys
    float scale;                      // times log2(e)
    int window;                       // 0: none
    int target, least, slots;         // workgroups a head of keys to split the cache over, steps of the shortest part, places for parts
    int vec;                          // out: groups of four values are aligned
};

// ------------------------------------------------------------------ what a workgroup does

// Sequence s as the split sees it.
struct SeqWork {
    int first, n, len;  // its first new token, how many, its length
    int base, steps;    // first position of the walk (a multiple of 16), steps of 32 from there
    int tiles, seq;
};

__device__ __forceinline__ int lane_of(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ int wave_total(int v) { return lane_of(wave_scan(v), 63); }

__device__ __forceinline__ SeqWork seq_work(const AttendArgs& a, int s, int rows) {
    SeqWork w;
    w.seq = s;
    int end;
    kv_segment(a.p, s, w.first, end);
    w.n = end - w.first;
    w.len = max(a.p.lens[s], 0);
    const int last = (int)min((int64_t)w.len, (int64_t)a.p.max_pages * a.p.page_size);
    w.base = a.window > 0 && w.len - w.n >= a.window ? (w.len - w.n - a.window + 1) & ~15 : 0;
    w.steps = w.n > 0 && last > w.base ? (last - w.base + kAtStep - 1) / kAtStep : 0;
    w.tiles = (int)(((int64_t)w.n * a.group + rows - 1) / rows);
    return w;
}

__device__ __forceinline__ SeqWork lane_work(const AttendArgs& a, int s, int rows) {
    return s < a.p.nseq ? seq_work(a, s, rows) : SeqWork{0, 0, 0, 0, 0, 0, 0};
}

// Steps of a part: the whole work over the target, at least `least`.
__device__ __forceinline__ int part_steps(const AttendArgs& a, int64_t work) {
    const int64_t c = (work + a.target - 1) / a.target;
    return (int)min(max(c, (int64_t)a.least), (int64_t)1 << 28);
}

__device__ __forceinline__ int parts_of(const SeqWork& w, int c) { return w.n > 0 ? max(1, (w.steps + c - 1) / c) : 0; }

struct Item {
    SeqWork w;
    int tile, part, parts, c;
    int slot;  // of its tile's part 0, where there are several parts
};

// Item i of the call's: every sequence's tiles of rows times its parts, in order.  False past the last.  Every
// wave finds it by itself.
__device__ __forceinline__ bool find_item(const AttendArgs& a, int i, int rows, Item& it) {
    const int lane = threadIdx.x & 63, nseq = a.p.nseq;
    if (a.plan) {
        // c, then for each sequence the items before it, and all of them; the same of the slots
        const int32_t *items = a.plan + 1, *slots = items + nseq + 1;
        it.c = a.plan[0];
        if (i >= items[nseq]) return false;
        const int stride = (nseq + 63) / 64;
        int s = stride * __popcll(__ballot(items[min((lane + 1) * stride, nseq)] <= i));
        const int end = min(s + stride, nseq);
        int more = 0;
        for (int j = s; j < end; j += 64) more += __popcll(__ballot(j + lane < end && items[min(j + lane + 1, nseq)] <= i));
        s = __builtin_amdgcn_readfirstlane(s + more);
        it.w = seq_work(a, s, rows);
        it.parts = parts_of(it.w, it.c);
        it.slot = slots[s];
        i -= items[s];
    } else {
        SeqWork w;
        int64_t work = 0;
        for (int j = 0; j < nseq; j += 64) {
            w = lane_work(a, j + lane, rows);
            const int64_t mine = (int64_t)w.steps * w.tiles;  // below 2^49 in all: two sums that fit 32 bits
            work += ((int64_t)wave_total((int)(mine >> 24)) << 24) + wave_total((int)(mine & 0xFFFFFF));
        }
        it.c = part_steps(a, work);
        int before = 0, slots = 0;
        bool found = false;
        for (int j = 0; j < nseq && !found; j += 64) {
            if (nseq > 64) w = lane_work(a, j + lane, rows);
            const int parts = parts_of(w, it.c), mine = parts * w.tiles, slot = parts > 1 ? mine : 0;
            const int upto = wave_scan(mine), sl = wave_scan(slot), total = lane_of(upto, 63);
            if (i < before + total) {
                const int s = __popcll(__ballot(before + upto <= i));
                it.w.first = lane_of(w.first, s);
                it.w.n = lane_of(w.n, s);
                it.w.len = lane_of(w.len, s);
                it.w.base = lane_of(w.base, s);
                it.w.steps = lane_of(w.steps, s);
                it.w.tiles = lane_of(w.tiles, s);
                it.w.seq = j + s;
                it.parts = lane_of(parts, s);
                it.slot = slots + lane_of(sl - slot, s);
                i -= before + lane_of(upto - mine, s);
                found = true;
            }
            before += total;
            slots += lane_of(sl, 63);
        }
        if (!found) return false;
    }
    it.tile = i / it.parts;
    it.part = i - it.tile * it.parts;
    it.slot += it.tile * it.parts;
    return true;
}

// ------------------------------------------------------------------ values as the matrix instructions take them

template <int TYPE, int NB>
struct Side {
    static constexpr int kFactor = TYPE == kKvF16 ? 64 * NB : TYPE == kKvQ8 ? 32 * NB : 16 * NB;  // bytes of a position
    static constexpr int kScale = TYPE == kKvF16 ? 0 : 2 * NB;
    static constexpr int kRow = kFactor + kScale;
};

// N bytes from an address of any alignment, the last dword filled up with zeros.
template <int N>
__device__ __forceinline__ void load_bytes(uint32_t* w, const char* p) {
    if constexpr (N % 4) w[N / 4] = 0;
    __builtin_memcpy(w, p, N);
}

// (u - 128) 2^-10 of two biased bytes, which perm lays into the low bytes of two halves: as binary16 they are u 2^-24.
__device__ __forceinline__ uint32_t biased_pair(uint32_t x) {
    const half2_t scale = {(_Float16)16384.0f, (_Float16)16384.0f}, bias = {(_Float16)-0.125f, (_Float16)-0.125f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(half2_t, x), scale, bias));
}
constexpr uint32_t pair_sel(int low, int high) { return 0x0C000C00u | (uint32_t)low | (uint32_t)high << 16; }

// Biased levels of a dword of index bytes, the low halves' and the high halves'.
__device__ __forceinline__ void levels(uint32_t q, uint32_t& lo, uint32_t& hi) {
    lo = iq4nl_lookup_u(q & 0x07070707u, ((q >> 1) & 0x04040404u) | 0x03020100u);
    hi = iq4nl_lookup_u((q >> 4) & 0x07070707u, ((q >> 5) & 0x04040404u) | 0x03020100u);
}

__device__ __forceinline__ half8_t as_half8(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return __builtin_bit_cast(half8_t, u32x4{x, y, z, w}); }

// The keys of 16 positions: lane (position n, quarter g) holds of every block b the eight dims 32b + 16i + 4g +
// (0..3), i = 0, 1 (binary16: 32b + 8g + (0..7)).
template <int TYPE, int NB>
struct Keys {
    static constexpr int kBytes = TYPE == kKvF16 ? 0 : Side<TYPE, NB>::kFactor / 4;
    uint32_t w[TYPE == kKvF16 ? 4 * NB : kBytes / 4];
    uint32_t d[TYPE == kKvF16 ? 1 : 2 * NB];  // scales [position 4g + r][block], two a dword

    __device__ __forceinline__ void load(const char* chunk, int place, int page_size) {
        const int n = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
        if constexpr (TYPE == kKvF16) {
            const char* p = chunk + (uint32_t)((place + n) * (64 * NB) + 16 * g);
#pragma unroll
            for (int b = 0; b < NB; ++b) __builtin_memcpy(w + 4 * b, __builtin_assume_aligned(p + 64 * b, 16), 16);
        } else {
            load_bytes<kBytes>(w, chunk + (uint32_t)((place + n) * Side<TYPE, NB>::kFactor + g * kBytes));
            load_bytes<8 * NB>(d, chunk + (uint32_t)(page_size * Side<TYPE, NB>::kFactor + (place + 4 * g) * (2 * NB)));
        }
    }
    // Biases the bytes of q8_0, looks the levels of iq4_nl up.
    struct Ready {
        uint32_t a[TYPE == kKvF16 ? 4 * NB : kBytes / 4], b[TYPE == kKvIq4 ? kBytes / 4 : 1];
    };
    __device__ __forceinline__ void ready(Ready& r) const {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(w) / 4); ++i) {
            if constexpr (TYPE == kKvF16) r.a[i] = w[i];
            else if constexpr (TYPE == kKvQ8) r.a[i] = w[i] ^ 0x80808080u;
            else levels(w[i], r.a[i], r.b[i]);
        }
    }
    __device__ static __forceinline__ half8_t block(const Ready& r, int b) {
        if constexpr (TYPE == kKvF16) return as_half8(r.a[4 * b], r.a[4 * b + 1], r.a[4 * b + 2], r.a[4 * b + 3]);
        uint32_t x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (TYPE == kKvQ8) {
                const int at = (m * NB + b) * 2;
                x[m] = biased_pair(perm(r.a[at / 4], r.a[at / 4], pair_sel(at % 4, at % 4 + 1)));
            } else {
                const int at = m * NB + b;
                x[m] = biased_pair(perm(r.b[at / 4], r.a[at / 4], pair_sel(at % 4, at % 4 + 4)));
            }
        }
        return as_half8(x[0], x[1], x[2], x[3]);
    }
    __device__ __forceinline__ float scale(int r, int b) const {
        const int i = r * NB + b;
        return (float)__builtin_bit_cast(half2_t, d[i / 2])[i & 1];
    }
};

__device__ __forceinline__ bool not_finite(uint32_t half) { return (half & 0x7C00u) == 0x7C00u; }

// The values of 32 positions: lane (n, g) holds, of the positions 4g .. 4g+3 of both halves, the dims that
// row n of the 2 NB operands V^T takes: tile (b, i) dim 32b + 16i + n (binary16: tile j dim 2 NB n + j).
template <int TYPE, int NB>
struct Values {
    static constexpr int kBytes = Side<TYPE, NB>::kFactor / 16;
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[8][kWords];
    uint32_t d[2][TYPE == kKvF16 ? 1 : 2 * NB];  // scales [half][position 4g + r][block]

    __device__ __forceinline__ void load(int half, const char* chunk, int place, int page_size) {
        const int n = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
        const char* p = chunk + (uint32_t)((place + 4 * g) * Side<TYPE, NB>::kFactor + n * kBytes);
#pragma unroll
        for (int r = 0; r < 4; ++r) load_bytes<kBytes>(w[4 * half + r], p + r * Side<TYPE, NB>::kFactor);
        if constexpr (TYPE != kKvF16)
            load_bytes<8 * NB>(d[half], chunk + (uint32_t)(page_size * Side<TYPE, NB>::kFactor + (place + 4 * g) * (2 * NB)));
    }
    __device__ __forceinline__ _Float16 scale(int x, int b) const {
        const int i = (x & 3) * NB + b;
        return __builtin_bit_cast(half2_t, d[x >> 2][i / 2])[i & 1];
    }
    // The binary16 bits of the largest magnitude among the scales, of all positions or of those seen.
    template <bool MASKED>
    __device__ __forceinline__ int largest(int seen) const {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 most = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                uint32_t v = d[h][i] & 0x7FFF7FFFu;
                if constexpr (MASKED) {
                    const int x = 4 * h + 2 * i / NB, y = 4 * h + (2 * i + 1) / NB;
                    if (x == y) v = seen >> x & 1 ? v : 0u;
                    else v = (seen >> x & 1 ? v & 0xFFFFu : 0u) | (seen >> y & 1 ? v & 0xFFFF0000u : 0u);
                }
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, v));
            }
        return max((int)most.x, (int)most.y);
    }
    // Scales that are not finite: whether there are any, the blocks (bits) where a position seen has one, and without them.
    __device__ __forceinline__ bool any_odd() const {
        bool odd = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) odd |= not_finite(d[h][i]) || not_finite(d[h][i] >> 16);
        return odd;
    }
    __device__ __forceinline__ int odd_blocks(int seen) const {
        int blocks = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int b = 0; b < NB; ++b)
                blocks |= seen >> x & 1 && not_finite(__builtin_bit_cast(uint16_t, scale(x, b))) ? 1 << b : 0;
        return blocks;
    }
    // The scales as they are loaded, two a register, also past a branch that may change them.
    __device__ __forceinline__ void keep_words() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) asm("" : "+v"(d[h][i]));
    }
    __device__ __forceinline__ void drop_odd() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                const uint32_t v = d[h][i];
                d[h][i] = (not_finite(v) ? 0u : v & 0xFFFFu) | (not_finite(v >> 16) ? 0u : v & 0xFFFF0000u);
            }
    }
    // Biased bytes; of iq4_nl the levels, where two half dwords of neighbouring positions share a lookup.
    struct Ready {
        uint32_t a[8][kWords], b[TYPE == kKvIq4 ? 8 : 1][kWords];
    };
    __device__ __forceinline__ void ready(Ready& r) const {
#pragma unroll
        for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (TYPE == kKvF16) r.a[x][i] = w[x][i];
                else if constexpr (TYPE == kKvQ8) r.a[x][i] = w[x][i] ^ 0x80808080u;
                else if (kBytes % 4 != 2 || i < kWords - 1) levels(w[x][i], r.a[x][i], r.b[x][i]);
                else if (x & 1) {
                    levels(w[x - 1][i] | w[x][i] << 16, r.a[x - 1][i], r.b[x - 1][i]);
                    r.a[x][i] = r.a[x - 1][i];
                    r.b[x][i] = r.b[x - 1][i];
                }
            }
    }
    __device__ static __forceinline__ half8_t tile(const Ready& r, int t) {
        uint32_t o[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (TYPE == kKvF16) {
                o[m] = perm(r.a[2 * m + 1][t / 2], r.a[2 * m][t / 2], t & 1 ? 0x07060302u : 0x05040100u);
            } else if constexpr (TYPE == kKvQ8) {
                o[m] = biased_pair(perm(r.a[2 * m + 1][t / 4], r.a[2 * m][t / 4], pair_sel(t % 4, t % 4 + 4)));
            } else {
                const int b = t / 2, i = b / 4, shared = kBytes % 4 == 2 && i == kWords - 1 ? 2 : 0;
                const uint32_t lo = t & 1 ? r.b[2 * m][i] : r.a[2 * m][i], hi = t & 1 ? r.b[2 * m + 1][i] : r.a[2 * m + 1][i];
                o[m] = biased_pair(perm(hi, lo, pair_sel(b % 4, b % 4 + 4 + shared)));
            }
        }
        return as_half8(o[0], o[1], o[2], o[3]);
    }
    // The dim of row m of tile t.
    __device__ static __forceinline__ int dim(int t, int m) { return TYPE == kKvF16 ? 2 * NB * m + t : 16 * t + m; }
};

// Constants that the compiler does not see through: a product and sum with them stays one v_fma_mix_f32, which
// takes binary16 factors as they are; a plain difference or product would convert them first.
struct Mix {
    float minus, zero;
    __device__ __forceinline__ Mix() : minus(-1.0f), zero(0.0f) { asm("" : "+s"(minus), "+s"(zero)); }
    __device__ __forceinline__ float product(float x, _Float16 h) const { return __builtin_fmaf((float)h, x, zero); }
    __device__ __forceinline__ float rest(float x, _Float16 h) const { return __builtin_fmaf((float)h, minus, x); }
};

// Two binary16 parts of pairs of values: the nearest, and the nearest of what is left.
__device__ __forceinline__ void two_parts(const Mix& mix, float x, float y, uint32_t& hi, uint32_t& lo) {
    const half2_t h = __builtin_convertvector((float2_t{x, y}), half2_t);
    const float2_t rest = {mix.rest(x, h.x), mix.rest(y, h.y)};
    hi = __builtin_bit_cast(uint32_t, h);
    lo = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, half2_t));
}

// Maximum and sum over the lanes n, n + 16, n + 32, n + 48.
__device__ __forceinline__ float rows_max(float v) {
    const int x = __builtin_bit_cast(int, v);
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_fmaxf(__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1]));
    const int y = __builtin_bit_cast(int, v);
    r = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (int)r[0]), __builtin_bit_cast(float, (int)r[1]));
}
__device__ __forceinline__ float rows_sum(float v) {
    const int x = __builtin_bit_cast(int, v);
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
    const int y = __builtin_bit_cast(int, v);
    r = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return __builtin_bit_cast(float, (int)r[0]) + __builtin_bit_cast(float, (int)r[1]);
}

// Orders LDS accesses of the lanes of a wave, which run in step.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int rows_or(int v) {
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = (int)r[0] | (int)r[1];
    r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (int)r[0] | (int)r[1];
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float power(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

__device__ __forceinline__ void store4(const float* v, void* p, int64_t i, int type, int vec) {
    if (vec && type == kF32) {
        *(float4_t*)((float*)p + i) = float4_t{v[0], v[1], v[2], v[3]};
    } else if (vec) {
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = type == kBin16 ? f2h(v[e]) : f2bf(v[e]);
        *(u32x2*)((uint16_t*)p + i) = u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) store_value(p, i + e, type, v[e]);
    }
}

// Four dims of row r (of its sequence's) of a head of keys, and with the first of them the row's lse.
__device__ __forceinline__ void write_row(const AttendArgs& a, int first, int head, int r, int d, float4_t f, float most, float sum) {
    const int token = r / a.group, h = head * a.group + r - token * a.group;
    const float v[4] = {f[0], f[1], f[2], f[3]};
    store4(v, a.out, (first + token) * a.ldo + (int64_t)h * a.p.dim + d, a.otype, a.vec);
    if (d == 0 && a.lse)
        a.lse[(int64_t)(first + token) * a.nheads + h] = sum != 0.0f ? most * 0.693147180559945f + __logf(sum) : -INFINITY;
}

// The weight of a result whose maximum is m beside one of a maximum `top`.  At m = -inf its sums are zeros, or NaN.
__device__ __forceinline__ float beside(float m, float top) { return m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top); }

// Floats of a slot and head.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }

// ------------------------------------------------------------------ the pass

// Resources: the queries' parts lie in LDS, read again each step (two 16-byte reads a block), which leaves the
// registers to the keys and values in flight.
template <int KT, int VT, int NB, int RT>
__global__ __launch_bounds__(64 * kAtWaves, 2) void attend_kernel(AttendArgs a) {
    constexpr int kRows = 16 * RT, kDim = 32 * NB, kTiles = 2 * NB;
    constexpr bool kKeyBlocks = KT != kKvF16, kValBlocks = VT != kKvF16;
    // The next keys are read before the weights, or after the values where the registers do not hold both.
    constexpr bool kEarly = NB < 8;
    // The sums of two waves at a time, at the end; until then a quarter is a wave's own for odd values.
    __shared__ __attribute__((aligned(16))) float so[2][kRows][kDim + 4];
    __shared__ float lm[2][kRows], ll[2][kRows], lc[kRows];
    static_assert(sizeof(so) / kAtWaves >= kRows * kAtStep * 4 + kDim * 2, "weights and a position's values");
    __shared__ __attribute__((aligned(16))) uint32_t lq[RT][NB][2][64][4];
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = (int)(blockIdx.x % (uint32_t)a.p.nheads);
    Item it;
    if (!find_item(a, (int)(blockIdx.x / (uint32_t)a.p.nheads), kRows, it)) return;
    const SeqWork& w = it.w;

    // The rows of the tile: lane n's, the positions [rlo, rhi) that they see, and the same over all of them.
    const int row0 = it.tile * kRows, rows = min(kRows, w.n * a.group - row0), cap = a.p.max_pages * a.p.page_size;
    const auto low = [&](int pos) { return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0; };
    const int tok0 = row0 / a.group, tok1 = (row0 + rows - 1) / a.group;
    const int pos0 = w.len - w.n + tok0, pos1 = w.len - w.n + tok1;
    const int lo_min = low(pos0), lo_max = low(pos1), hi_min = min(pos0 + 1, cap), hi_max = min(pos1 + 1, cap);

    // This wave's steps of the part, those that the tile sees.
    int s0 = it.part * it.c, s1 = min(s0 + it.c, w.steps);
    s0 = max(s0, (lo_min - w.base) / kAtStep);
    s1 = min(s1, (hi_max - w.base + kAtStep - 1) / kAtStep);  // (hi_max below 0: none)
    const int ksteps = s1 > s0 + wave ? (s1 - s0 - wave + kAtWaves - 1) / kAtWaves : 0;
    const int start = w.base + kAtStep * (s0 + wave);
    const Mix mix;
    const int64_t kchunk = (int64_t)head * a.p.page_size * Side<KT, NB>::kRow, vchunk = (int64_t)head * a.p.page_size * Side<VT, NB>::kRow;
    int pages = 0, places = 0;  // lane 2 i + half: the page of step i (of 32) and the place in it
    const auto read_pages = [&](int k) {
        const int pos = start + kAtStep * kAtWaves * (k + (lane >> 1)) + 16 * (lane & 1);
        const bool in = k + (lane >> 1) < ksteps;
        pages = in ? kv_page(a.p, w.seq, pos) : -1;
        places = in ? (int)((uint32_t)pos % (uint32_t)a.p.page_size) : 0;
    };
    // A position that does not exist is read at page 0 and not seen.
    Keys<KT, NB> keys[2];
    const auto load_keys = [&](int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pg = lane_of(pages, 2 * (k & 31) + h);
            keys[h].load(a.k.base + (pg < 0 ? 0 : pg * a.k.stride) + kchunk, lane_of(places, 2 * (k & 31) + h), a.p.page_size);
        }
    };
    if (ksteps > 0) {
        read_pages(0);
        load_keys(0);
    }

    // The queries, 16 threads a row: scaled, their two parts laid out as the operand that a lane reads.
    // Thread j holds the dims 32b + j and 32b + 16 + j (element 2m + i of a block format's operand is dim 32b + 16i
    // + 4g + m) or 32b + 2j and the next (binary16: element e is 32b + 8g + e).
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int r = 16 * x + (int)threadIdx.x / 16, j = threadIdx.x & 15, tok = (row0 + r) / a.group;
        const bool live = r < rows;
        const int64_t at = live ? (w.first + tok) * a.ldq + (int64_t)(head * a.group + row0 + r - tok * a.group) * kDim : 0;
        float v[NB][2], most = 0.0f;
        if (a.qtype == kF32) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) v[b][i] = ((const float*)a.q)[at + 32 * b + (kKeyBlocks ? 16 * i + j : 2 * j + i)];
        } else {
            uint32_t raw[NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) raw[b][i] = ((const uint16_t*)a.q)[at + 32 * b + (kKeyBlocks ? 16 * i + j : 2 * j + i)];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) v[b][i] = a.qtype == kBin16 ? h2f(raw[b][i]) : bf2f(raw[b][i]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[b][i] = live ? v[b][i] * a.scale : 0.0f;
                most = __builtin_fmaxf(most, __builtin_fabsf(v[b][i]));
            }
        most = __builtin_fmaxf(most, dpp<0xB1>(most));
        most = __builtin_fmaxf(most, dpp<0x4E>(most));
        most = __builtin_fmaxf(most, dpp<0x141>(most));
        most = __builtin_fmaxf(most, dpp<0x140>(most));
        // the power of two that puts the largest in [2^13, 2^14); rows of nothing but tiny values stay what they are
        const int e = min(max((int)(__builtin_bit_cast(uint32_t, most) >> 23), 40), 254) - 126;
        const float up = power(14 - e);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t hi, lo;
            two_parts(mix, v[b][0] * up, v[b][1] * up, hi, lo);
            lq[x][b][0][16 * (j / 4) + r % 16][j % 4] = hi;
            lq[x][b][1][16 * (j / 4) + r % 16][j % 4] = lo;
        }
        if (j == 0) lc[r] = power(e - 14 + (kKeyBlocks ? 10 : 0));
    }
    __syncthreads();

    int rlo[RT], rhi[RT];
    float c[RT];  // scores are c times the sums of the scaled operands
    float4_t o[RT][kTiles];
    float m[RT], l[RT], limit[RT], fold[RT];
    int bound[RT];  // the binary16 bits of limit, a power of two above the scales of values that the row has seen
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        const int r = 16 * x + n;
        const int pos = w.len - w.n + (row0 + r) / a.group;
        rlo[x] = low(pos);
        rhi[x] = r < rows ? min(pos + 1, cap) : 0;
        c[x] = lc[r];
        m[x] = -INFINITY;
        l[x] = 0.0f;
        limit[x] = power(-24);
        fold[x] = power(14 + 24);
        bound[x] = 1;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[x][t] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const auto queries = [&](int x, int b, int part) { return __builtin_bit_cast(half8_t, *(const u32x4*)lq[x][b][part][lane]); };

    for (int k = 0; k < ksteps; ++k) {
        const int j0 = start + kAtStep * kAtWaves * k;
        const bool exist[2] = {lane_of(pages, 2 * (k & 31)) >= 0, lane_of(pages, 2 * (k & 31) + 1) >= 0};
        Values<VT, NB> vals;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pg = lane_of(pages, 2 * (k & 31) + h);
            vals.load(h, a.v.base + (pg < 0 ? 0 : pg * a.v.stride) + vchunk, lane_of(places, 2 * (k & 31) + h), a.p.page_size);
        }
        float z[RT][8];
        {
            typename Keys<KT, NB>::Ready ready[2];
            keys[0].ready(ready[0]);
            keys[1].ready(ready[1]);
            float4_t s[RT][2], t[RT][2];
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[x][h] = t[x][h] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int r = 0; r < 4; ++r) z[x][4 * h + r] = 0.0f;
                }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (kKeyBlocks) __builtin_amdgcn_sched_barrier(0);
                const half8_t kb[2] = {Keys<KT, NB>::block(ready[0], b), Keys<KT, NB>::block(ready[1], b)};
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    const half8_t qh = queries(x, b, 0), ql = queries(x, b, 1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (kKeyBlocks) {
                            float4_t u = {0.0f, 0.0f, 0.0f, 0.0f};
                            u = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], ql, u, 0, 0, 0);
                            u = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], qh, u, 0, 0, 0);
#pragma unroll
                            for (int r = 0; r < 4; ++r) z[x][4 * h + r] = __builtin_fmaf(u[r], keys[h].scale(r, b), z[x][4 * h + r]);
                        } else {
                            s[x][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], qh, s[x][h], 0, 0, 0);
                            t[x][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kb[h], ql, t[x][h], 0, 0, 0);
                        }
                    }
                }
            }
            if constexpr (!kKeyBlocks) {
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[x][i] = s[x][i / 4][i & 3] + t[x][i / 4][i & 3];
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (kEarly && k + 1 < ksteps) {
            if ((k & 31) == 31) read_pages(k + 1);
            load_keys(k + 1);
        }
        // Positions that some row of the tile does not see: their scores go, whatever they are.  (The empty asm keeps
        // this a branch that steps in the middle of a cache skip.)
        const bool masked = j0 < lo_max || j0 + kAtStep > hi_min || !exist[0] || !exist[1];
        int seen[RT], most[RT];  // bit i of seen: position i of z
        if (masked) {
            asm volatile("");
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                seen[x] = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
                    const bool in = exist[i >> 2] && j >= rlo[x] && j < rhi[x];
                    seen[x] |= in ? 1 << i : 0;
                    z[x][i] = in ? z[x][i] : -INFINITY;
                }
            }
        }
        float top[RT];
        bool grew = false;
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            top[x] = m[x];
#pragma unroll
            for (int i = 0; i < 8; ++i) top[x] = __builtin_fmaxf(top[x], z[x][i]);
            top[x] = rows_max(top[x]);
            grew |= top[x] > m[x];
        }
        if (__any(grew)) {
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                const float shrink = top[x] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((m[x] - top[x]) * c[x]);
                m[x] = top[x];
                l[x] *= shrink;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) o[x][t] *= shrink;
            }
        }
        // Weights: of binary16 values times 2^14; of blocks' to be multiplied by the scales and a power of two that
        // keeps the largest product there.
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const float from = m[x] == -INFINITY ? 0.0f : __builtin_fmaf(-m[x], c[x], kValBlocks ? 0.0f : 14.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[x][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[x][i], c[x], from));
                l[x] += z[x][i];
            }
        }
        if constexpr (kValBlocks) {
            bool above = false;
            vals.keep_words();
            if (masked) {
                asm volatile("");
#pragma unroll
                for (int x = 0; x < RT; ++x) most[x] = vals.template largest<true>(seen[x]);
                // A scale that is not finite must not meet the weight 0 of a row that does not see it: it is left
                // out, and makes its block NaN in the rows that do.
                if (__any(vals.any_odd())) {
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        const int blocks = rows_or(vals.odd_blocks(seen[x]));
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
                            if (blocks >> (t / 2) & 1) o[x][t] = float4_t{NAN, NAN, NAN, NAN};
                    }
                    vals.drop_odd();
                }
            } else {
#pragma unroll
                for (int x = 0; x < RT; ++x) most[x] = x ? most[0] : vals.template largest<false>(0);
            }
            vals.keep_words();
#pragma unroll
            for (int x = 0; x < RT; ++x) above |= most[x] >= bound[x];
            if (__any(above)) {
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    const float d = rows_max(__builtin_fabsf(h2f(min(most[x], 0x7C00))));  // (an infinity, NaN: 2^17)
                    const int e = max(min((int)(__builtin_bit_cast(uint32_t, d) >> 23) - 126, 17), -24);
                    const float to = __builtin_fmaxf(limit[x], power(e)), shrink = limit[x] * (1.0f / to);
                    limit[x] = to;
                    fold[x] = 16384.0f / to;
                    bound[x] = to > 65536.0f ? 0x10000 : (int)f2h(to);
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) o[x][t] *= shrink;
                }
            }
        } else if (masked) {
            asm volatile("");
            // Places that no row sees count as zeros.  Infinities and NaN that some rows see and others do not
            // must not meet the others' zeros in the products: they are added one position at a time, and left out there.
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = j0 + 16 * (i >> 2) + 4 * g + (i & 3);
                const bool some = exist[i >> 2] && j >= lo_min && j < hi_max;
#pragma unroll
                for (int e = 0; e < Values<VT, NB>::kWords; ++e) {
                    vals.w[i][e] = some ? vals.w[i][e] : 0u;
                    odd |= not_finite(vals.w[i][e]) || not_finite(vals.w[i][e] >> 16);
                }
            }
            if (__any(odd)) {
                float* weight = &so[0][0][0] + wave * (int)(sizeof(so) / 4 / kAtWaves);
                uint32_t* row = (uint32_t*)(weight + kRows * kAtStep);
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) weight[(16 * x + n) * kAtStep + 16 * (i >> 2) + 4 * g + (i & 3)] = seen[x] >> i & 1 ? z[x][i] : -1.0f;
                for (int u = 0; u < kAtStep; ++u) {
                    if (g == u / 4 % 4) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i == 4 * (u / 16) + u % 4)
#pragma unroll
                                for (int e = 0; e < Values<VT, NB>::kWords; ++e) row[n * Values<VT, NB>::kWords + e] = vals.w[i][e];
                    }
                    wave_fence();
#pragma unroll
                    for (int x = 0; x < RT; ++x) {
                        const float p = weight[(16 * x + n) * kAtStep + u];
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const uint32_t v = ((const uint16_t*)row)[Values<VT, NB>::dim(t, 4 * g + r)];
                                if (p >= 0.0f && not_finite(v)) o[x][t][r] += p * h2f(v);
                            }
                    }
                    wave_fence();
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < Values<VT, NB>::kWords; ++e) {
                        const uint32_t v = vals.w[i][e];
                        vals.w[i][e] = (not_finite(v) ? 0u : v & 0xFFFFu) | (not_finite(v >> 16) ? 0u : v & 0xFFFF0000u);
                    }
            }
        }
        if constexpr (kValBlocks) {
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) z[x][i] *= fold[x];
        }
        // The sums of values.
        typename Values<VT, NB>::Ready ready;
        vals.ready(ready);
        half8_t ph[RT], pl[RT];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            if (kValBlocks ? t % 2 == 0 : t == 0) {
                if constexpr (kValBlocks) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int x = 0; x < RT; ++x) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float u[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            u[e] = z[x][2 * i + e];
                            if constexpr (kValBlocks) u[e] = mix.product(u[e], vals.scale(2 * i + e, t / 2));
                        }
                        two_parts(mix, u[0], u[1], hi[i], lo[i]);
                    }
                    ph[x] = as_half8(hi[0], hi[1], hi[2], hi[3]);
                    pl[x] = as_half8(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            const half8_t v = Values<VT, NB>::tile(ready, t);
#pragma unroll
            for (int x = 0; x < RT; ++x) {
                o[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pl[x], o[x][t], 0, 0, 0);
                o[x][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, ph[x], o[x][t], 0, 0, 0);
            }
        }
        if (!kEarly && k + 1 < ksteps) {
            if ((k & 31) == 31) read_pages(k + 1);
            load_keys(k + 1);
        }
    }

    // The waves' results, in base-2 units of the scores: two waves to the other two through LDS, then those.
#pragma unroll
    for (int x = 0; x < RT; ++x) {
        l[x] = rows_sum(l[x]) * (kValBlocks ? 1.0f : power(-14));
        m[x] *= c[x];
        const float back = kValBlocks ? limit[x] * power(10 - 14) : power(-14);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) o[x][t] *= back;
    }
    const auto put = [&](int at) {
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            if (g == 0) {
                lm[at][16 * x + n] = m[x];
                ll[at][16 * x + n] = l[x];
            }
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) so[at][16 * x + n][Values<VT, NB>::dim(t, 4 * g + r)] = o[x][t][r];
        }
    };
    __syncthreads();
    if (wave >= 2) put(wave - 2);
    __syncthreads();
    if (wave < 2) {
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            const float other = lm[wave][16 * x + n], most = __builtin_fmaxf(m[x], other), mine = beside(m[x], most), its = beside(other, most);
            m[x] = most;
            l[x] = l[x] * mine + ll[wave][16 * x + n] * its;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) o[x][t][r] = o[x][t][r] * mine + so[wave][16 * x + n][Values<VT, NB>::dim(t, 4 * g + r)] * its;
        }
        put(wave);
    }
    __syncthreads();
    const bool whole = it.parts == 1;
    if (!whole && (it.slot < 0 || it.slot + it.part >= a.slots)) return;  // offsets that decrease: no place for it
    float* part = a.parts + ((int64_t)(it.slot + it.part) * a.p.nheads + head) * part_floats(kRows, kDim);
    for (int i = threadIdx.x; i < rows * (kDim / 4); i += 64 * kAtWaves) {
        const int r = i / (kDim / 4), d = 4 * (i - r * (kDim / 4));
        const float most = __builtin_fmaxf(lm[0][r], lm[1][r]), e0 = beside(lm[0][r], most), e1 = beside(lm[1][r], most);
        const float sum = e0 * ll[0][r] + e1 * ll[1][r];
        float4_t f = e0 * *(const float4_t*)&so[0][r][d] + e1 * *(const float4_t*)&so[1][r][d];
        if (whole) {
            f *= sum != 0.0f ? 1.0f / sum : 0.0f;
            write_row(a, w.first, head, row0 + r, d, f, most, sum);
        } else {
            if (d == 0) {
                part[r] = most;
                part[kRows + r] = sum;
            }
            *(float4_t*)(part + 2 * kRows + r * kDim + d) = f;
        }
    }
}

// The launch of one pair of formats, instantiated in a source of its own per format of the keys.
template <int KT, int VT>
void attend_pair(const AttendArgs& a, unsigned grid, int rt, hipStream_t st) {
    const dim3 block(64 * kAtWaves);
    switch (a.p.dim / 32 * 2 + rt) {
        case 5: hipLaunchKernelGGL((attend_kernel<KT, VT, 2, 1>), dim3(grid), block, 0, st, a); break;
        case 6: hipLaunchKernelGGL((attend_kernel<KT, VT, 2, 2>), dim3(grid), block, 0, st, a); break;
        case 7: hipLaunchKernelGGL((attend_kernel<KT, VT, 3, 1>), dim3(grid), block, 0, st, a); break;
        case 8: hipLaunchKernelGGL((attend_kernel<KT, VT, 3, 2>), dim3(grid), block, 0, st, a); break;
        case 9: hipLaunchKernelGGL((attend_kernel<KT, VT, 4, 1>), dim3(grid), block, 0, st, a); break;
        case 10: hipLaunchKernelGGL((attend_kernel<KT, VT, 4, 2>), dim3(grid), block, 0, st, a); break;
        case 13: hipLaunchKernelGGL((attend_kernel<KT, VT, 6, 1>), dim3(grid), block, 0, st, a); break;
        default: hipLaunchKernelGGL((attend_kernel<KT, VT, 8, 1>), dim3(grid), block, 0, st, a); break;
    }
}
void attend_f16(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);
void attend_q8(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);
void attend_iq4(const AttendArgs& a, unsigned grid, int rt, hipStream_t st);

}  // namespace qmm
