// qmm_norm.hip -- root-mean-square norm with the residual's addition and a q8_1 output, and the
// values of q8_1 blocks, for gfx950.
//
// r = x + res, y = r / sqrt(mean r^2 + eps) * w, all in binary32, in one pass over the row; r and y
// are rounded once when stored, yq holds q8_1(y) of the binary32 y.
#include "qmm_values.h"

namespace qmm {

struct NormArgs {
    const void *x, *res;
    void *res_out, *y;
    uint8_t* yq;
    const float* w;
    int64_t ldx, ldr, ldro, ldy;
    int64_t ntok;
    int hidden, xtype, rtype, ytype;
    float eps;
};

// Sum over aligned groups of L lanes (16, 32 or 64), in every lane: within rows of 16 by DPP, then
// across them by lane exchanges.
template <int L>
__device__ __forceinline__ float lanes_total(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    if constexpr (L >= 32) v += __shfl_xor(v, 16, 64);
    if constexpr (L >= 64) v += __shfl_xor(v, 32, 64);
    return v;
}

// Sum over the workgroup, each wave's total through LDS in wave order.
__device__ __forceinline__ float workgroup_total(float v) {
    __shared__ float part[16];
    v = lanes_total<64>(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
    for (unsigned w = 1; w < blockDim.x / 64; ++w) v += part[w];
    return v;
}

__device__ __forceinline__ char* at(void* p, int64_t row, int64_t ld, int type) {
    return (char*)p + row * ld * (type == kF32 ? 4 : 2);
}
__device__ __forceinline__ const char* at(const void* p, int64_t row, int64_t ld, int type) {
    return (const char*)p + row * ld * (type == kF32 ? 4 : 2);
}

// q8_1 of a block held by the four lanes of a quad, eight values each: quantize_lanes32's arithmetic
// (the maximum and the integer sum are exact in any order).
__device__ __forceinline__ void quantize_quad(const float* v, uint8_t* blk) {
    float amax = __builtin_fabsf(v[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[e]));
    amax = __builtin_fmaxf(amax, dpp<0xB1>(amax));
    amax = __builtin_fmaxf(amax, dpp<0x4E>(amax));
    const float d = amax / 127.0f;
    const bool zero = amax == 0.0f || d == 0.0f;
    int q[8], sum = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int r = round_away(v[e] / d);
        q[e] = zero ? 0 : r > 127 ? 127 : r < -127 ? -127 : r;
        sum += q[e];
    }
    sum += dpp_i<0xB1>(sum);
    sum += dpp_i<0x4E>(sum);
    uint32_t* o = (uint32_t*)blk;
    const int p = threadIdx.x & 3;
    if (p == 0) o[0] = zero ? 0u : (f2h(d) | (f2h(opaque(d * (float)sum)) << 16));
    o[1 + 2 * p] = (q[0] & 255) | ((q[1] & 255) << 8) | ((q[2] & 255) << 16) | ((uint32_t)q[3] << 24);
    o[2 + 2 * p] = (q[4] & 255) | ((q[5] & 255) << 8) | ((q[6] & 255) << 16) | ((uint32_t)q[7] << 24);
}

// A row in registers: thread i of its `threads` holds the 8-value pieces i, i + threads, ... (NV of
// them), read and written 16 bytes at a time.  L = 0: one workgroup per row, NV = 1 up to 8192 values
// (8192 x 2560, binary32 + binary16 in, two binary16 out: 38.2 us, 5.5 TB/s; with a wave per row and
// NV = 5 41 us).  L = 16, 32, 64: rows of up to 8 L values, L lanes each.  Every load is issued
// before the first is used; a piece past the row is read at its start and counts as zeros.
// Bound: bytes; few rows: the launch and one load, one sum, one store after another.
template <int NV, int L>
__global__ __launch_bounds__(L ? 256 : 1024) void rmsnorm_kernel(NormArgs a) {
    const int threads = L ? L : (int)blockDim.x, tid = L ? (int)threadIdx.x % (L ? L : 1) : (int)threadIdx.x;
    const int64_t t = L ? (int64_t)blockIdx.x * (256 / (L ? L : 1)) + threadIdx.x / (L ? L : 1) : blockIdx.x;
    if (L && t >= a.ntok) return;
    const char* x = at(a.x, t, a.ldx, a.xtype);
    Raw8 xr[NV], rr[NV], wr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = 8 * (tid + threads * i);
        load_raw8(xr[i], x, j < a.hidden ? j : 0, a.xtype);
    }
    if (a.res) {
        const char* res = at(a.res, t, a.ldr, a.rtype);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = 8 * (tid + threads * i);
            load_raw8(rr[i], res, j < a.hidden ? j : 0, a.rtype);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = 8 * (tid + threads * i);
        load_raw8(wr[i], a.w, j < a.hidden ? j : 0, kF32);
    }
    float r[NV][8], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        unpack8(xr[i], a.xtype, r[i]);
        if (a.res) {
            float v[8];
            unpack8(rr[i], a.rtype, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] += v[e];
        }
        const int j = 8 * (tid + threads * i);
        if (j >= a.hidden) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[i][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s += r[i][e] * r[i][e];
    }
    if (a.res_out) {
        char* ro = at(a.res_out, t, a.ldro, a.rtype);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = 8 * (tid + threads * i);
            if (j < a.hidden) store8(ro, j, a.rtype, r[i]);
        }
    }
    float total;
    if constexpr (L) total = lanes_total<L>(s);
    else total = workgroup_total(s);
    const float rstd = 1.0f / sqrtf(total / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float w[8];
        unpack8(wr[i], kF32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = r[i][e] * rstd * w[e];
    }
    if (a.y) {
        char* y = at(a.y, t, a.ldy, a.ytype);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = 8 * (tid + threads * i);
            if (j < a.hidden) store8(y, j, a.ytype, r[i]);
        }
    }
    if (a.yq) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = 8 * (tid + threads * i);
            if (j < a.hidden) quantize_quad(r[i], a.yq + (t * (a.hidden / 32) + j / 32) * 36);
        }
    }
}

// q8_1 of blocks held one value a lane; every lane of the wave calls it.
__device__ __forceinline__ void store_lane_block(const NormArgs& a, int64_t t, int j, bool in, float y) {
    uint32_t hdr;
    const int q = quantize_lanes32(y, hdr);
    const uint32_t word = pack4_lanes(q);
    uint32_t* dst = (uint32_t*)(a.yq + (t * (a.hidden / 32) + j / 32) * 36);
    if (in && j % 32 == 0) dst[0] = hdr;
    if (in && j % 4 == 0) dst[1 + j % 32 / 4] = word;
}

// The same for rows of any width and alignment: thread i holds the values i, i + blockDim.x, ... (NE
// of them), read and written one at a time, neighbouring lanes at neighbouring values; 32 consecutive
// lanes hold one q8_1 block.  Bound: the narrow loads and stores; 517 x 1001 bfloat16 3.4 us, 8192 x
// 2561 binary16 (84 MB) 45 us, where 2560 take 15.7 in 16-byte pieces.
template <int NE>
__global__ __launch_bounds__(1024) void rmsnorm_any_kernel(NormArgs a) {
    const int threads = (int)blockDim.x, tid = (int)threadIdx.x;
    const int64_t t = blockIdx.x;
    const char* x = at(a.x, t, a.ldx, a.xtype);
    float r[NE], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int j = tid + threads * i;
        r[i] = load_value(x, j < a.hidden ? j : 0, a.xtype);
    }
    if (a.res) {
        const char* res = at(a.res, t, a.ldr, a.rtype);
        float v[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int j = tid + threads * i;
            v[i] = load_value(res, j < a.hidden ? j : 0, a.rtype);
        }
#pragma unroll
        for (int i = 0; i < NE; ++i) r[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        if (tid + threads * i >= a.hidden) r[i] = 0.0f;
        s += r[i] * r[i];
    }
    if (a.res_out) {
        char* ro = at(a.res_out, t, a.ldro, a.rtype);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int j = tid + threads * i;
            if (j < a.hidden) store_value(ro, j, a.rtype, r[i]);
        }
    }
    const float rstd = 1.0f / sqrtf(workgroup_total(s) / (float)a.hidden + a.eps);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int j = tid + threads * i;
        r[i] = r[i] * rstd * a.w[j < a.hidden ? j : 0];
    }
    if (a.y) {
        char* y = at(a.y, t, a.ldy, a.ytype);
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int j = tid + threads * i;
            if (j < a.hidden) store_value(y, j, a.ytype, r[i]);
        }
    }
    if (a.yq) {
#pragma unroll
        for (int i = 0; i < NE; ++i) store_lane_block(a, t, tid + threads * i, tid + threads * i < a.hidden, r[i]);
    }
}

// Long rows of any alignment (a row would not fit the registers one value at a time): x and res are
// read twice, each value written by the thread that read it last, so in-place outputs are safe.  2048 x
// 12289 binary16 (101 MB) 76 us, where 12288 take 23.9 in 16-byte pieces.
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs a) {
    const int64_t t = blockIdx.x;
    const char *x = at(a.x, t, a.ldx, a.xtype), *res = a.res ? at(a.res, t, a.ldr, a.rtype) : nullptr;
    const auto value = [&](int j) {
        const float v = load_value(x, j, a.xtype);
        return res ? v + load_value(res, j, a.rtype) : v;
    };
    float s = 0.0f;
    for (int j = threadIdx.x; j < a.hidden; j += 1024) {
        const float r = value(j);
        s += r * r;
    }
    const float rstd = 1.0f / sqrtf(workgroup_total(s) / (float)a.hidden + a.eps);
    for (int j0 = 0; j0 < a.hidden; j0 += 1024) {
        const int j = j0 + (int)threadIdx.x;
        const bool in = j < a.hidden;
        const float r = in ? value(j) : 0.0f, y = in ? r * rstd * a.w[j] : 0.0f;
        if (in && a.res_out) store_value(at(a.res_out, t, a.ldro, a.rtype), j, a.rtype, r);
        if (in && a.y) store_value(at(a.y, t, a.ldy, a.ytype), j, a.ytype, y);
        if (a.yq) store_lane_block(a, t, j, in, y);
    }
}

// One thread per 4 values of a block (a dword of the block).  Bound: a launch at 1 x 2560 (2.0 us); 8192 x
// 2560 to binary16 15.9 us (66 MB, 4.1 TB/s), to binary32 28.5 us (107 MB, 3.8 TB/s), four stores a thread.
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

#include "qmm_types.h"

using namespace qmm;

constexpr int64_t kNormMaxRows = (1 << 22) - 1;  // a workgroup of 1024 threads a row, below 2^32 threads
constexpr int64_t kValuesMaxBlocks = ((int64_t)1 << 29) - 32;  // 8 threads a block, whole workgroups of 256, below 2^32 threads

extern "C" int qmm_rmsnorm(int xtype, const void* x, int64_t ldx, int rtype, const void* res, int64_t ldr, void* res_out,
                           int64_t ldro, const float* w, float eps, int64_t ntok, int64_t hidden, int ytype, void* y,
                           int64_t ldy, void* yq, void* stream) {
    if (!valid_type(xtype) || ntok < 0 || hidden < 1 || ldx < hidden || !(eps >= 0.0f) || !(eps <= 3.4e38f)) return QMM_EINVAL;
    if ((res || res_out) && !valid_type(rtype)) return QMM_EINVAL;
    if (res && ldr < hidden) return QMM_EINVAL;
    if (res_out && ldro < hidden) return QMM_EINVAL;
    if (y && (!valid_type(ytype) || ldy < hidden)) return QMM_EINVAL;
    if (yq && hidden % 32) return QMM_EINVAL;
    if (hidden > kMaxK || ntok > kNormMaxRows) return QMM_EUNSUPPORTED;
    if (ntok == 0) return QMM_OK;
    if (!x || !w || (!y && !yq && !res_out)) return QMM_EINVAL;
    if (!aligned(x, type_bytes(xtype)) || !aligned(w, 4) || !aligned(yq, 4) || (y && !aligned(y, type_bytes(ytype))) ||
        (res && !aligned(res, type_bytes(rtype))) || (res_out && !aligned(res_out, type_bytes(rtype))))
        return QMM_EALIGN;
    NormArgs a{x, res, res_out, y, (uint8_t*)yq, w, ldx, ldr, ldro, ldy, ntok, (int)hidden, xtype, rtype, ytype, eps};
    const hipStream_t st = as_stream(stream);
    const auto rows16 = [](const void* p, int64_t ld, int type) { return aligned(p, 16) && ld * (int64_t)type_bytes(type) % 16 == 0; };
    if (hidden % 8 == 0 && aligned(w, 16) && rows16(x, ldx, xtype) && (!res || rows16(res, ldr, rtype)) &&
        (!res_out || rows16(res_out, ldro, rtype)) && (!y || rows16(y, ldy, ytype))) {
        const int pieces = (int)(hidden / 8);
        if (pieces <= 64) {
            const int lanes = pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
            const dim3 grid((unsigned)((ntok * lanes + 255) / 256));
            if (lanes == 16) hipLaunchKernelGGL((rmsnorm_kernel<1, 16>), grid, dim3(256), 0, st, a);
            else if (lanes == 32) hipLaunchKernelGGL((rmsnorm_kernel<1, 32>), grid, dim3(256), 0, st, a);
            else hipLaunchKernelGGL((rmsnorm_kernel<1, 64>), grid, dim3(256), 0, st, a);
            return launch_status();
        }
        const int nv = pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : 4;
        const dim3 grid((unsigned)ntok), block(64 * ((pieces + 64 * nv - 1) / (64 * nv)));
        if (nv == 1) hipLaunchKernelGGL((rmsnorm_kernel<1, 0>), grid, block, 0, st, a);
        else if (nv == 2) hipLaunchKernelGGL((rmsnorm_kernel<2, 0>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((rmsnorm_kernel<4, 0>), grid, block, 0, st, a);
        return launch_status();
    }
    const dim3 grid((unsigned)ntok);
    if (hidden <= 4096)
        hipLaunchKernelGGL(rmsnorm_any_kernel<4>, grid, dim3((unsigned)((hidden + 255) / 256) * 64), 0, st, a);
    else if (hidden <= 8192)
        hipLaunchKernelGGL(rmsnorm_any_kernel<8>, grid, dim3((unsigned)((hidden + 511) / 512) * 64), 0, st, a);
    else
        hipLaunchKernelGGL(rmsnorm_long_kernel, grid, dim3(1024), 0, st, a);
    return launch_status();
}

extern "C" int qmm_dequantize_q8_1(const void* xq, int64_t k, int64_t ncols, int otype, void* out, int64_t ldo, void* stream) {
    if (k < 32 || k % 32 || ncols < 0 || ldo < k || (otype != QMM_TYPE_F32 && otype != QMM_TYPE_F16)) return QMM_EINVAL;
    if (k > (int64_t)1 << 30 || ncols > (int64_t)1 << 31 || ncols * (k / 32) > kValuesMaxBlocks) return QMM_EUNSUPPORTED;
    if (ncols == 0) return QMM_OK;
    if (!xq || !out) return QMM_EINVAL;
    if (!aligned(xq, 4) || !aligned(out, type_bytes(otype))) return QMM_EALIGN;
    const int64_t nblk = ncols * (k / 32);
    hipLaunchKernelGGL(dequantize_q8_1_kernel, dim3((unsigned)((nblk * 8 + 255) / 256)), dim3(256), 0, as_stream(stream),
                       (const uint8_t*)xq, (int)(k / 32), nblk, otype, out, ldo);
    return launch_status();
}
