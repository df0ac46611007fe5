// decode_device.cuh -- device helpers that the decode step's operators share: rounding to
// the 16-bit types and to E4M3, and sizes that several go by.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace qmv {

// Two values rounded to the 16-bit type, a in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Four values, none above 448 in magnitude, rounded to E4M3 (ties to even), a in the lowest
// byte. NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

constexpr int kSms = 152;
constexpr int kScaleTokens = 16;   // consecutive places of a cache of codes that share a scale, for each head

}  // namespace qmv
