// qmm_lora.hip -- low-rank adapters of many requests beside a shared projection, for gfx950:
// y[t] = base[t] + scale_i * B_i (A_i x[t]), i the adapter of the token's segment.
//
// Two launches, each over tiles of the tokens of one segment (found by a scan of the segments, so
// their lengths stay on the device): the inner values v = A_i x[t] in binary32 into the workspace,
// then the outer product added to the base.
#include "qmm_values.h"

namespace qmm {

constexpr int kLoraMaxRank = 256;

struct LoraArgs {
    const void* x;
    const uint16_t *a, *b;
    const int32_t *ranks, *seg_off, *seg_adapter;
    const float *scales, *base;
    float *y, *v;
    int64_t ldx, ldbase, ldy;
    int ntok, k, nadapters, max_rank, nseg, nrows, split;
};

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct LoraTile {
    int t0, nt, adapter, rank;  // nt = 0: no such tile
};

// Tile `tile` of the segments' tiles of T tokens each (the last of a segment holds what is left):
// its tokens [t0, t0 + nt) and their adapter, -1 for none.  Every lane of the wave calls it.
__device__ __forceinline__ LoraTile find_tile(const LoraArgs& a, int T, int tile) {
    const int l = threadIdx.x & 63;
    for (int s0 = 0; s0 < a.nseg; s0 += 64) {
        const int s = s0 + l;
        int o0 = 0, o1 = 0, i = -1;
        if (s < a.nseg) {
            o0 = a.seg_off[s];
            o1 = a.seg_off[s + 1];
            i = a.seg_adapter[s];
        }
        o0 = o0 < 0 ? 0 : o0 > a.ntok ? a.ntok : o0;
        o1 = o1 < o0 ? o0 : o1 > a.ntok ? a.ntok : o1;
        int end = (o1 - o0 + T - 1) / T;
        const int n = end;
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(end, d, 64);
            if (l >= d) end += u;
        }
        const uint64_t past = __ballot(end > tile);
        if (past) {
            const int src = (int)__builtin_ctzll(past);
            LoraTile r;
            r.t0 = __builtin_amdgcn_readlane(o0, src) + (tile - __builtin_amdgcn_readlane(end - n, src)) * T;
            const int left = __builtin_amdgcn_readlane(o1, src) - r.t0;
            r.nt = left < T ? left : T;
            r.adapter = __builtin_amdgcn_readlane(i, src);
            if (r.adapter < 0 || r.adapter >= a.nadapters) r.adapter = -1;
            r.rank = r.adapter < 0 ? 0 : a.ranks[r.adapter];
            r.rank = r.rank < 0 ? 0 : r.rank > a.max_rank ? a.max_rank : r.rank;
            return r;
        }
        tile -= __builtin_amdgcn_readlane(end, 63);
    }
    return {0, 0, -1, 0};
}

// ------------------------------------------------------------------ inner values

// One step of 32 columns: 8 values of x for each of MT token rows, 8 values of A for each of NR
// rank rows; lane l holds row l % 16 and columns 8 (l / 16) .. + 7 of the step.
template <int XT, int NR, int MT>
struct DownStep {
    u32x4 x[MT][XT == kF32 ? 2 : 1];
    u32x4 a[NR];
};

// Workgroup (tile, split): W waves over the tile's 16 MT tokens and 16 NR rank rows, each wave a run
// of the split's 32-column steps, summed through LDS in wave order.  Rows past the tile or the rank
// read the last valid row; their sums are not stored (or stored as 0).
template <int XT, int NR, int MT, int W>
__global__ __launch_bounds__(64 * W) void lora_down_kernel(LoraArgs a) {
    constexpr int T = 16 * MT, R = 16 * NR, U = NR <= 4 ? 4 : 2;
    __shared__ float part[W][T][R + 1];
    const LoraTile tile = find_tile(a, T, blockIdx.x);
    if (tile.nt == 0 || tile.rank == 0) return;
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, row = l & 15, q = l >> 4;
    const char* xr[MT];
    const uint16_t* ar[NR];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int t = 16 * m + row;
        xr[m] = (const char*)a.x + ((int64_t)(tile.t0 + (t < tile.nt ? t : tile.nt - 1)) * a.ldx + 8 * q) * (XT == kF32 ? 4 : 2);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int j = 16 * n + row;
        ar[n] = a.a + ((int64_t)tile.adapter * a.max_rank + (j < tile.rank ? j : tile.rank - 1)) * a.k + 8 * q;
    }
    const int steps = a.k / 32, runs = W * a.split;
    const int per = (steps + runs - 1) / runs;
    const int c0 = ((int)blockIdx.y * W + w) * per, c1 = c0 + per < steps ? c0 + per : steps;

    f32x4 acc[MT][NR];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[m][n] = f32x4{};

    auto load = [&](DownStep<XT, NR, MT>& s, int c) {
        c = c < c1 ? c : c1 - 1;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const u32x4* p = (const u32x4*)(xr[m] + (int64_t)c * (XT == kF32 ? 128 : 64));
            s.x[m][0] = p[0];
            if constexpr (XT == kF32) s.x[m][1] = p[1];
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) s.a[n] = *(const u32x4*)(ar[n] + (int64_t)c * 32);
    };
    auto apply = [&](const DownStep<XT, NR, MT>& s) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const half8 b = __builtin_bit_cast(half8, s.a[n]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (XT == kF32) {
                    const f32x4 x0 = __builtin_bit_cast(f32x4, s.x[m][0]), x1 = __builtin_bit_cast(f32x4, s.x[m][1]);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(e < 4 ? x0[e] : x1[e - 4], (float)b[e], acc[m][n], 0, 0, 0);
                } else {
                    acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, s.x[m][0]), b, acc[m][n], 0, 0, 0);
                }
            }
        }
    };
    if (c0 < c1) {
        for (int c = c0; c < c1; c += U) {
            DownStep<XT, NR, MT> s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) load(s[u], c + u);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u < c1) apply(s[u]);
        }
    }
    // accumulator register r of lane l: token 4 (l / 16) + r, rank row l % 16
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) part[w][16 * m + 4 * q + r][16 * n + row] = acc[m][n][r];
    __syncthreads();
    float* v = a.v + ((int64_t)blockIdx.y * a.ntok + tile.t0) * a.max_rank;
    for (int i = threadIdx.x; i < tile.nt * R; i += 64 * W) {
        const int t = i / R, j = i % R;
        float s = part[0][t][j];
#pragma unroll
        for (int u = 1; u < W; ++u) s += part[u][t][j];
        if (j < a.max_rank) v[(int64_t)t * a.max_rank + j] = j < tile.rank ? s : 0.0f;
    }
}

// ------------------------------------------------------------------ outer product

constexpr int kUpRows = 256;  // rows of y per workgroup: 4 waves of two 32-row blocks

// Workgroup (row block, tile): NT blocks of 32 tokens by 256 rows of y.  The inner values (the sum
// of the splits) are scaled per token by the power of two that puts the largest into [512, 1024)
// and cut into binary16 high and low parts, v = hi + lo to 2^-24 of the largest, so the product
// with B runs on binary16 MFMA with nothing lost to range: acc = hi B + lo B, y = base +
// acc * (scale 2^e).
template <int NT>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
    constexpr int T = 32 * NT, G = 256 / T;  // G threads per token in the prologue
    constexpr int MAXG = 4;                  // 8-rank groups per thread there
    extern __shared__ u32x4 frag[];          // [hi, lo][step][half][token]
    __shared__ uint32_t largest[T];
    __shared__ float factor[T];
    const LoraTile tile = find_tile(a, T, blockIdx.y);
    if (tile.nt == 0) return;
    const int tid = threadIdx.x, w = tid >> 6, l = tid & 63, col = l & 31, h = l >> 5;
    const int r0 = (int)blockIdx.x * kUpRows;
    const float* base = a.base + (int64_t)tile.t0 * a.ldbase + r0;
    float* y = a.y + (int64_t)tile.t0 * a.ldy + r0;
    const int rows = a.nrows - r0 < kUpRows ? a.nrows - r0 : kUpRows;
    if (tile.rank == 0) {  // no adapter: y = base
        if (base == y && a.ldbase == a.ldy) return;
        if (tid < rows)
            for (int t = 0; t < tile.nt; ++t) y[t * a.ldy + tid] = base[t * a.ldbase + tid];
        return;
    }
    const int steps = (tile.rank + 15) / 16;

    // base: register r of token block n, row block c: token 32 n + 8 (r / 4) + 4 h + r % 4
    float in[NT][2][16];
    const bool full = tile.nt == T && rows == kUpRows;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = 32 * n + 8 * (r / 4) + 4 * h + r % 4, j = 64 * w + 32 * c + col;
                in[n][c][r] = full || (t < tile.nt && j < rows) ? base[t * a.ldbase + j] : 0.0f;
            }

    // inner values -> high and low parts
    const int tok = tid % T, g0 = tid / T;
    float v[MAXG][8];
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < MAXG; ++i) {
        const int j = 8 * (g0 + G * i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        if (tok < tile.nt && j < tile.rank) {
            for (int s = 0; s < a.split; ++s) {
                const f32x4* p = (const f32x4*)(a.v + ((int64_t)s * a.ntok + tile.t0 + tok) * a.max_rank + j);
                const f32x4 lo = p[0], hi = p[1];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] += e < 4 ? lo[e] : hi[e - 4];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __builtin_bit_cast(uint32_t, v[i][e]) & 0x7FFFFFFFu;
                if (b < 0x7F800000u && b > big) big = b;  // infinities and NaN keep to themselves
            }
        }
    }
    if (tid < T) largest[tid] = 0;
    __syncthreads();
    atomicMax(&largest[tok], big);
    __syncthreads();
    // the largest is in [2^ex, 2^(ex+1)) or subnormal; no scaling where there is no finite one but 0
    const int ex = largest[tok] ? (int)(largest[tok] >> 23) - 127 : 9;
    if (tid < T) factor[tid] = ldexpf(a.scales[tile.adapter], ex - 9);
    const int part = steps * 2 * T;
#pragma unroll
    for (int i = 0; i < MAXG; ++i) {
        const int g = g0 + G * i;
        if (g < 2 * steps) {
            half8 hi, lo;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = ldexpf(v[i][e], 9 - ex);
                hi[e] = (_Float16)s;
                lo[e] = __builtin_isfinite(s) ? (_Float16)(s - (float)hi[e]) : (_Float16)0.0f;
            }
            frag[g * T + tok] = __builtin_bit_cast(u32x4, hi);
            frag[part + g * T + tok] = __builtin_bit_cast(u32x4, lo);
        }
    }
    __syncthreads();

    f32x16 acc[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[n][c] = f32x16{};
    const uint16_t* br[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int j = 64 * w + 32 * c + col;
        br[c] = a.b + ((int64_t)tile.adapter * a.nrows + r0 + (j < rows ? j : rows - 1)) * a.max_rank;
    }
    for (int s = 0; s < steps; ++s) {
        const int j = 16 * s + 8 * h;
        half8 b[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            b[c] = *(const half8*)(br[c] + (j < a.max_rank ? j : 0));
            if (16 * s + 16 > tile.rank) {  // columns past the rank may hold anything
#pragma unroll
                for (int e = 0; e < 8; ++e) b[c][e] = j + e < tile.rank ? b[c][e] : (_Float16)0.0f;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const half8 hi = __builtin_bit_cast(half8, frag[(2 * s + h) * T + 32 * n + col]);
            const half8 lo = __builtin_bit_cast(half8, frag[part + (2 * s + h) * T + 32 * n + col]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                acc[n][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(lo, b[c], acc[n][c], 0, 0, 0);
                acc[n][c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(hi, b[c], acc[n][c], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int t = 32 * n + 8 * (r / 4) + 4 * h + r % 4, j = 64 * w + 32 * c + col;
                if (full || (t < tile.nt && j < rows)) y[t * a.ldy + j] = in[n][c][r] + acc[n][c][r] * factor[t];
            }
}

}  // namespace qmm

#include "qmm_host.h"

using namespace qmm;

constexpr int64_t kLoraMaxTokens = 1 << 20;
constexpr int kLoraMaxSegments = 1 << 14;

// How many workgroups share the columns of one token tile: enough that few tiles still fill the GPU.
static int lora_split(int64_t ntok) { return ntok <= 64 ? 8 : ntok <= 1024 ? 2 : 1; }

extern "C" size_t qmm_lora_workspace(int64_t ntok, int max_rank) {
    if (ntok < 0 || ntok > kLoraMaxTokens || max_rank < 8 || max_rank % 8 || max_rank > kLoraMaxRank) return 0;
    return (size_t)lora_split(ntok) * ntok * max_rank * 4 + 16;
}

template <int XT>
static void launch_down(const LoraArgs& p, hipStream_t st) {
    const auto grid = [&](int T) { return dim3((unsigned)(p.ntok / T + p.nseg), (unsigned)p.split); };
    if (p.max_rank <= 16) hipLaunchKernelGGL((lora_down_kernel<XT, 1, 2, 8>), grid(32), dim3(512), 0, st, p);
    else if (p.max_rank <= 32) hipLaunchKernelGGL((lora_down_kernel<XT, 2, 2, 8>), grid(32), dim3(512), 0, st, p);
    else if (p.max_rank <= 64) hipLaunchKernelGGL((lora_down_kernel<XT, 4, 2, 4>), grid(32), dim3(256), 0, st, p);
    else if (p.max_rank <= 128) hipLaunchKernelGGL((lora_down_kernel<XT, 8, 1, 4>), grid(16), dim3(256), 0, st, p);
    else hipLaunchKernelGGL((lora_down_kernel<XT, 16, 1, 2>), grid(16), dim3(128), 0, st, p);
}

extern "C" int qmm_lora(int xtype, const void* x, int64_t ldx, int64_t ntok, int64_t k, const uint16_t* a, const uint16_t* b,
                        const int32_t* ranks, const float* scales, int nadapters, int max_rank, const int32_t* seg_off,
                        const int32_t* seg_adapter, int nseg, const float* base, int64_t ldbase, float* y, int64_t ldy,
                        int64_t nrows, void* ws, size_t ws_bytes, void* stream) {
    if ((xtype != QMM_TYPE_F16 && xtype != QMM_TYPE_F32) || ntok < 0 || k < 32 || k % 32 || ldx < k || nadapters < 1 || max_rank < 8 ||
        max_rank % 8 || nseg < 0 || nrows < 1 || ldbase < nrows || ldy < nrows)
        return QMM_EINVAL;
    if (k > kMaxK || max_rank > kLoraMaxRank || ntok > kLoraMaxTokens || nseg > kLoraMaxSegments || nrows > 0x7FFFFF00) return QMM_EUNSUPPORTED;
    if (ntok == 0 || nseg == 0) return QMM_OK;
    if (!x || !a || !b || !ranks || !scales || !seg_off || !seg_adapter || !base || !y || !ws) return QMM_EINVAL;
    if (base == y && ldbase != ldy) return QMM_EINVAL;
    if (!aligned(x, 16) || ldx * (int64_t)type_bytes(xtype) % 16 || !aligned(a, 16) || !aligned(b, 16) || !aligned(ranks, 4) ||
        !aligned(scales, 4) || !aligned(seg_off, 4) || !aligned(seg_adapter, 4) || !aligned(base, 4) || !aligned(y, 4) || !aligned(ws, 16))
        return QMM_EALIGN;
    if (ws_bytes < qmm_lora_workspace(ntok, max_rank)) return QMM_ESPACE;
    LoraArgs p{x, a, b, ranks, seg_off, seg_adapter, scales, base, y, (float*)ws, ldx, ldbase, ldy, (int)ntok, (int)k,
               nadapters, max_rank, nseg, (int)nrows, lora_split(ntok)};
    const hipStream_t st = as_stream(stream);
    if (xtype == QMM_TYPE_F32) launch_down<kF32>(p, st);
    else launch_down<kBin16>(p, st);
    const unsigned rowblocks = (unsigned)((nrows + kUpRows - 1) / kUpRows);
    const size_t lds = (size_t)((max_rank + 15) / 16) * 64;  // hi and lo fragments per token
    if (max_rank <= 128 && ntok >= 32 * (int64_t)nseg)
        hipLaunchKernelGGL(lora_up_kernel<2>, dim3(rowblocks, (unsigned)(ntok / 64 + nseg)), dim3(256), lds * 64, st, p);
    else
        hipLaunchKernelGGL(lora_up_kernel<1>, dim3(rowblocks, (unsigned)(ntok / 32 + nseg)), dim3(256), lds * 32, st, p);
    return launch_status();
}
