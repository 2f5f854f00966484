// qmm_values.h -- tensor values of the norm, routing and adapter kernels: binary32, binary16 and
// bfloat16 elements read as binary32 and written with one rounding to nearest even.
#pragma once

#include "qmm_device.h"

namespace qmm {

enum : int { kF32 = 1, kBin16 = 2, kBf16 = 3 };  // QMM_TYPE_*

// binary32 -> bfloat16, round to nearest even; a NaN stays a NaN.
__device__ __forceinline__ uint32_t f2bf(float f) {
    const uint32_t u = __builtin_bit_cast(uint32_t, f);
    if (f != f) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ float bf2f(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }

__device__ __forceinline__ float load_value(const void* p, int64_t i, int type) {
    if (type == kF32) return ((const float*)p)[i];
    const uint32_t b = ((const uint16_t*)p)[i];
    return type == kBin16 ? h2f(b) : bf2f(b);
}
__device__ __forceinline__ void store_value(void* p, int64_t i, int type, float v) {
    if (type == kF32) ((float*)p)[i] = v;
    else ((uint16_t*)p)[i] = (uint16_t)(type == kBin16 ? f2h(v) : f2bf(v));
}

// Inclusive scan over the wave: rows of 16 lanes by DPP shifts, the rows by the broadcasts of each
// row's (then each half's) last lane.
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2, 3
    return v;
}

// Eight consecutive values as loaded: 16 bytes of a 16-bit type, 32 of binary32.
struct Raw8 {
    u32x4 a, b;
};
// i: element index of the first, a multiple of 8 from a 16-byte aligned row start.
__device__ __forceinline__ void load_raw8(Raw8& r, const void* row, int i, int type) {
    if (type == kF32) {
        r.a = *(const u32x4*)((const float*)row + i);
        r.b = *(const u32x4*)((const float*)row + i + 4);
    } else {
        r.a = *(const u32x4*)((const uint16_t*)row + i);
    }
}
__device__ __forceinline__ void unpack8(const Raw8& r, int type, float* v) {
    const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
    if (type == kF32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(float, e < 4 ? a[e] : b[e - 4]);
    } else if (type == kBin16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = h2f(a[e / 2] >> (16 * (e & 1)));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e & 1 ? __builtin_bit_cast(float, a[e / 2] & 0xFFFF0000u) : bf2f(a[e / 2]);
    }
}
__device__ __forceinline__ void store8(void* row, int i, int type, const float* v) {
    u32x4 o;
    if (type == kF32) {
        typedef float f4 __attribute__((ext_vector_type(4)));
        *(f4*)((float*)row + i) = f4{v[0], v[1], v[2], v[3]};
        *(f4*)((float*)row + i + 4) = f4{v[4], v[5], v[6], v[7]};
        return;
    }
    if (type == kBin16) {
        o.x = f2h(v[0]) | (f2h(v[1]) << 16);
        o.y = f2h(v[2]) | (f2h(v[3]) << 16);
        o.z = f2h(v[4]) | (f2h(v[5]) << 16);
        o.w = f2h(v[6]) | (f2h(v[7]) << 16);
    } else {
        o.x = f2bf(v[0]) | (f2bf(v[1]) << 16);
        o.y = f2bf(v[2]) | (f2bf(v[3]) << 16);
        o.z = f2bf(v[4]) | (f2bf(v[5]) << 16);
        o.w = f2bf(v[6]) | (f2bf(v[7]) << 16);
    }
    *(u32x4*)((uint16_t*)row + i) = o;
}

}  // namespace qmm
