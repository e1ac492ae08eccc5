// e4m3.cuh -- quantisation to 8 bits, shared by the kernels that write e4m3 codes
// and scales:  a = max(max |v|, 2^-100),  scale = a / 448,  q = e4m3(v * (448 / a)).
//
// NaN and infinities: the maxima are taken over the bit patterns of |v| as
// unsigned integers, where NaN is largest, so a NaN reaches the scale (and q).
#pragma once

#include "ffn_internal.cuh"

namespace ffn {

constexpr float kE4m3Max = 448.f;
constexpr int kE4m3Block = 128;   // columns (and rows, of a weight) of one scale

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// max(a, 2^-100) with NaN kept (both are bit patterns of non-negative floats)
__device__ __forceinline__ float floor_amax(float a) {
    const uint32_t b = __float_as_uint(a), lo = __float_as_uint(7.888609052210118e-31f);
    return __uint_as_float(b > lo ? b : lo);
}

// two values to e4m3 (lo in the low byte), nearest even, finite values clamped to +-448
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

}  // namespace ffn
