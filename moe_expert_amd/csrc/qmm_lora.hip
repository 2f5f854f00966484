// qmm_lora.hip -- low-rank adapters of many requests beside a shared projection, for gfx950:
// y[t] = base[t] + scale_i * B_i (A_i x[t]), i the adapter of the token's segment.
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
    int xtype, ntok, k, nadapters, max_rank, nseg, nrows;
};

// The adapter of token t: -1 for none, -2 where no segment holds the token.
__device__ __forceinline__ int adapter_of(const LoraArgs& a, int t) {
    for (int s = 0; s < a.nseg; ++s)
        if (t >= a.seg_off[s] && t < a.seg_off[s + 1]) {
            const int i = a.seg_adapter[s];
            return i >= 0 && i < a.nadapters ? i : -1;
        }
    return -2;
}
__device__ __forceinline__ int rank_of(const LoraArgs& a, int i) {
    const int r = a.ranks[i];
    return r < 0 ? 0 : r > a.max_rank ? a.max_rank : r;
}

// v[t][j] = A_i[j] . x[t]: one wave per (token, j).
__global__ __launch_bounds__(64) void lora_down_kernel(LoraArgs a) {
    const int t = blockIdx.x, j = blockIdx.y;
    const int i = adapter_of(a, t);
    float s = 0.0f;
    if (i >= 0 && j < rank_of(a, i)) {
        const uint16_t* row = a.a + ((int64_t)i * a.max_rank + j) * a.k;
        for (int c = threadIdx.x; c < a.k; c += 64) s += h2f(row[c]) * load_value(a.x, t * a.ldx + c, a.xtype);
    }
    for (int m = 32; m; m >>= 1) s += __shfl_xor(s, m, 64);
    if (threadIdx.x == 0) a.v[(int64_t)t * a.max_rank + j] = s;
}

// y[t][r] = base[t][r] + scale_i * B_i[r] . v[t]: one thread per (token, r).
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
    const int t = blockIdx.x, r = blockIdx.y * 256 + threadIdx.x;
    const int i = adapter_of(a, t);
    if (r >= a.nrows || i == -2) return;
    const float base = a.base[t * a.ldbase + r];
    float s = 0.0f;
    if (i >= 0) {
        const int rank = rank_of(a, i);
        const uint16_t* row = a.b + ((int64_t)i * a.nrows + r) * a.max_rank;
        for (int j = 0; j < rank; ++j) s += h2f(row[j]) * a.v[(int64_t)t * a.max_rank + j];
        s *= a.scales[i];
    }
    a.y[t * a.ldy + r] = base + s;
}

}  // namespace qmm

#include "qmm_host.h"

using namespace qmm;

extern "C" size_t qmm_lora_workspace(int64_t ntok, int max_rank) {
    if (ntok < 0 || ntok > 0x7FFFFFFF || max_rank < 8 || max_rank % 8 || max_rank > kLoraMaxRank) return 0;
    return (size_t)ntok * max_rank * 4 + 16;
}

extern "C" int qmm_lora(int xtype, const void* x, int64_t ldx, int64_t ntok, int64_t k, const uint16_t* a, const uint16_t* b,
                        const int32_t* ranks, const float* scales, int nadapters, int max_rank, const int32_t* seg_off,
                        const int32_t* seg_adapter, int nseg, const float* base, int64_t ldbase, float* y, int64_t ldy,
                        int64_t nrows, void* ws, size_t ws_bytes, void* stream) {
    if ((xtype != QMM_TYPE_F16 && xtype != QMM_TYPE_F32) || ntok < 0 || k < 32 || k % 32 || ldx < k || nadapters < 1 || max_rank < 8 ||
        max_rank % 8 || nseg < 0 || nrows < 1 || ldbase < nrows || ldy < nrows)
        return QMM_EINVAL;
    if (k > kMaxK || max_rank > kLoraMaxRank || ntok > 0x7FFFFFFF || nrows > 0x7FFFFFFF) return QMM_EUNSUPPORTED;
    if (ntok == 0 || nseg == 0) return QMM_OK;
    if (!x || !a || !b || !ranks || !scales || !seg_off || !seg_adapter || !base || !y || !ws) return QMM_EINVAL;
    if (base == y && ldbase != ldy) return QMM_EINVAL;
    if (!aligned(x, 16) || ldx * (int64_t)type_bytes(xtype) % 16 || !aligned(a, 16) || !aligned(b, 16) || !aligned(ranks, 4) ||
        !aligned(scales, 4) || !aligned(seg_off, 4) || !aligned(seg_adapter, 4) || !aligned(base, 4) || !aligned(y, 4) || !aligned(ws, 16))
        return QMM_EALIGN;
    if (ws_bytes < qmm_lora_workspace(ntok, max_rank)) return QMM_ESPACE;
    LoraArgs p{x, a, b, ranks, seg_off, seg_adapter, scales, base, y, (float*)ws, ldx, ldbase, ldy, xtype, (int)ntok, (int)k,
               nadapters, max_rank, nseg, (int)nrows};
    const hipStream_t st = as_stream(stream);
    hipLaunchKernelGGL(lora_down_kernel, dim3((unsigned)ntok, (unsigned)max_rank), dim3(64), 0, st, p);
    hipLaunchKernelGGL(lora_up_kernel, dim3((unsigned)ntok, (unsigned)((nrows + 255) / 256)), dim3(256), 0, st, p);
    return launch_status();
}
