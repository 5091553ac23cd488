// Shared by the paged 8-bit key/value cache kernels (coc_kv_append.cu,
// coc_kv_attention.cu): conversions and the scale rule.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "coc_internal.h"
#include "coc_kv_units.h"

namespace coc {
namespace {

// The least exponent a page's scale takes (an all-zero page would otherwise
// have none; 2^-100 keeps code * scale a normal fp32).
constexpr int kMinScaleExp = -100;

template <bool BF16>
__device__ __forceinline__ float to_float16bit(uint16_t v) {
    if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return __half2float(__ushort_as_half(v));
}

// Loads of what an earlier kernel on the stream may have written (see load_index).
__device__ __forceinline__ float load_float(const float* p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 load_float4(const float* p) {
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 load_uint4(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Least power of two s with amax <= 448 s, at least 2^kMinScaleExp.  amax =
// 1.f x 2^e gives 2^(e - 8) for 1.f <= 1.75 (448 = 1.75 x 2^8), else 2^(e - 7).
// A power of two makes x / s and a later change of scale exact up to e4m3's
// own underflow, and costs no precision: e4m3 is a floating-point type.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23) - 127;
    const int s = e - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>((s < kMinScaleExp ? kMinScaleExp : s) + 127) << 23);
}

}  // namespace
}  // namespace coc
