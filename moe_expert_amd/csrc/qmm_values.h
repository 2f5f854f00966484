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

}  // namespace qmm
