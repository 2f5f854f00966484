// qmm_norm.hip -- root-mean-square norm with the residual's addition and a q8_1 output, and the
// values of q8_1 blocks, for gfx950.
//
// r = x + res, y = r / sqrt(mean r^2 + eps) * w, all in binary32; r and y are rounded once when
// stored, yq holds q8_1(y) of the binary32 y.
#include "qmm_values.h"

namespace qmm {

struct NormArgs {
    const void *x, *res;
    void *res_out, *y;
    uint8_t* yq;
    const float* w;
    int64_t ldx, ldr, ldro, ldy;
    int hidden, xtype, rtype, ytype;
    float eps;
};

constexpr int kNormThreads = 256;

__device__ __forceinline__ float residual_value(const NormArgs& a, int64_t t, int j) {
    const float v = load_value(a.x, t * a.ldx + j, a.xtype);
    return a.res ? v + load_value(a.res, t * a.ldr + j, a.rtype) : v;
}

// One workgroup per row.  Lane order within a wave is value order, so 32 consecutive lanes hold one
// q8_1 block.
__global__ __launch_bounds__(kNormThreads) void rmsnorm_kernel(NormArgs a) {
    __shared__ float part[kNormThreads];
    const int64_t t = blockIdx.x;
    float s = 0.0f;
    for (int j = threadIdx.x; j < a.hidden; j += kNormThreads) {
        const float r = residual_value(a, t, j);
        s += r * r;
    }
    part[threadIdx.x] = s;
    __syncthreads();
    for (int n = kNormThreads / 2; n; n >>= 1) {
        if ((int)threadIdx.x < n) part[threadIdx.x] += part[threadIdx.x + n];
        __syncthreads();
    }
    const float rstd = 1.0f / sqrtf(part[0] / (float)a.hidden + a.eps);
    for (int j0 = 0; j0 < a.hidden; j0 += kNormThreads) {
        const int j = j0 + (int)threadIdx.x;
        const bool in = j < a.hidden;
        float r = 0.0f, y = 0.0f;
        if (in) {
            r = residual_value(a, t, j);
            y = r * rstd * a.w[j];
        }
        if (in && a.res_out) store_value(a.res_out, t * a.ldro + j, a.rtype, r);
        if (in && a.y) store_value(a.y, t * a.ldy + j, a.ytype, y);
        if (a.yq) {
            uint32_t hdr;
            const int q = quantize_lanes32(y, hdr);
            const uint32_t word = pack4_lanes(q);
            uint32_t* dst = (uint32_t*)(a.yq + (t * (a.hidden / 32) + j / 32) * 36);
            if (in && j % 32 == 0) dst[0] = hdr;
            if (in && j % 4 == 0) dst[1 + j % 32 / 4] = word;
        }
    }
}

// One thread per 4 values of a block.
__global__ __launch_bounds__(256) void dequantize_q8_1_kernel(const uint8_t* __restrict__ xq, int nb, int64_t nblk, int otype,
                                                              void* __restrict__ out, int64_t ldo) {
    const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t blk = g >> 3;
    if (blk >= nblk) return;
    const int i = (int)(g & 7);
    const uint32_t* b = (const uint32_t*)(xq + blk * 36);
    const float d = h2f(b[0]);
    const uint32_t q = b[1 + i];
    const int64_t c = blk / nb;
    const int64_t o = c * ldo + (blk - c * nb) * 32 + 4 * i;
    for (int e = 0; e < 4; ++e) store_value(out, o + e, otype, opaque(d * (float)(int8_t)(q >> (8 * e))));
}

}  // namespace qmm

#include "qmm_host.h"

using namespace qmm;

extern "C" int qmm_rmsnorm(int xtype, const void* x, int64_t ldx, int rtype, const void* res, int64_t ldr, void* res_out,
                           int64_t ldro, const float* w, float eps, int64_t ntok, int64_t hidden, int ytype, void* y,
                           int64_t ldy, void* yq, void* stream) {
    if (!valid_type(xtype) || ntok < 0 || hidden < 1 || ldx < hidden || !(eps >= 0.0f) || !(eps <= 3.4e38f)) return QMM_EINVAL;
    if ((res || res_out) && !valid_type(rtype)) return QMM_EINVAL;
    if (res && ldr < hidden) return QMM_EINVAL;
    if (res_out && ldro < hidden) return QMM_EINVAL;
    if (y && (!valid_type(ytype) || ldy < hidden)) return QMM_EINVAL;
    if (yq && hidden % 32) return QMM_EINVAL;
    if (hidden > kMaxK || ntok > 0x7FFFFFFF) return QMM_EUNSUPPORTED;
    if (ntok == 0) return QMM_OK;
    if (!x || !w || (!y && !yq && !res_out)) return QMM_EINVAL;
    if (!aligned(x, type_bytes(xtype)) || !aligned(w, 4) || !aligned(yq, 4) || (y && !aligned(y, type_bytes(ytype))) ||
        (res && !aligned(res, type_bytes(rtype))) || (res_out && !aligned(res_out, type_bytes(rtype))))
        return QMM_EALIGN;
    NormArgs a{x, res, res_out, y, (uint8_t*)yq, w, ldx, ldr, ldro, ldy, (int)hidden, xtype, rtype, ytype, eps};
    hipLaunchKernelGGL(rmsnorm_kernel, dim3((unsigned)ntok), dim3(kNormThreads), 0, as_stream(stream), a);
    return launch_status();
}

extern "C" int qmm_dequantize_q8_1(const void* xq, int64_t k, int64_t ncols, int otype, void* out, int64_t ldo, void* stream) {
    if (k < 32 || k % 32 || ncols < 0 || ldo < k || (otype != QMM_TYPE_F32 && otype != QMM_TYPE_F16)) return QMM_EINVAL;
    if (k > (int64_t)1 << 30 || ncols > (int64_t)1 << 31 || ncols * (k / 32) >= (int64_t)1 << 31) return QMM_EUNSUPPORTED;
    if (ncols == 0) return QMM_OK;
    if (!xq || !out) return QMM_EINVAL;
    if (!aligned(xq, 4) || !aligned(out, type_bytes(otype))) return QMM_EALIGN;
    const int64_t nblk = ncols * (k / 32);
    hipLaunchKernelGGL(dequantize_q8_1_kernel, dim3((unsigned)((nblk * 8 + 255) / 256)), dim3(256), 0, as_stream(stream),
                       (const uint8_t*)xq, (int)(k / 32), nblk, otype, out, ldo);
    return launch_status();
}
