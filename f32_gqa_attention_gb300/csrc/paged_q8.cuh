// paged_q8.cuh -- codes and scales of the 8-bit paged cache on the device.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged_q8.h"

namespace vtmu {

__device__ __forceinline__ float q8_nan_max(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float q8_abs_top(float t, const float4& x) {
    t = q8_nan_max(q8_nan_max(t, fabsf(x.x)), fabsf(x.y));
    return q8_nan_max(q8_nan_max(t, fabsf(x.z)), fabsf(x.w));
}

// A unit's scale and what its codes are formed with.
struct Q8Scale {
    float scale;  // NaN: an element is not finite
    float inv;    // 1 / scale (0 then): exact for a power of two
};
template <int FORM>
__device__ __forceinline__ Q8Scale q8_scale(float top) {
    constexpr float kLeast = 0x1p-126f;
    Q8Scale s;
    if constexpr (FORM == kFormInt8) {
        s.scale = fmaxf(top / 127.f, kLeast);
    } else {
        // top = 1.f 2^(E - 127); 448 = 1.75 2^8: the exponent E - 8, one more above 1.75.
        const uint32_t b = __float_as_uint(top);
        const int e = (int)(b >> 23) - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
        s.scale = __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
    }
    s.inv = 1.f / s.scale;
    if (!(top < __int_as_float(0x7f800000))) {
        s.scale = __int_as_float(0x7fc00000);
        s.inv = 0.f;
    }
    return s;
}

// The integer nearest to x / s, ties to even.  x inv is off by a rounding or two, so the
// integer r next to it may be off by one; the remainder x - r s is exact in an FMA (a
// multiple of the smaller operand's last place, at most s), and 2 |x - r s| against s
// says on which side the quotient lies.
__device__ __forceinline__ int q8_nearest(float x, const Q8Scale& s) {
    float r = rintf(x * s.inv);
    const float rest = fmaf(-r, s.scale, x), twice = 2.f * fabsf(rest);
    const bool odd = ((int)r & 1) != 0;
    if (twice > s.scale || (twice == s.scale && odd)) r += copysignf(1.f, rest);
    return (int)r;
}
template <int FORM>
__device__ __forceinline__ uint8_t q8_code(float x, const Q8Scale& s) {
    if constexpr (FORM == kFormInt8)
        return s.inv == 0.f ? 0 : (uint8_t)(int8_t)q8_nearest(x, s);
    else
        return s.inv == 0.f ? 0 : (uint8_t)__nv_cvt_float_to_fp8(x * s.inv, __NV_SATFINITE, __NV_E4M3);
}
template <int FORM>
__device__ __forceinline__ uint32_t q8_codes4(const float4& x, const Q8Scale& s) {
    if constexpr (FORM == kFormE4m3) {
        if (s.inv == 0.f) return 0;
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x * s.inv, x.y * s.inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z * s.inv, x.w * s.inv), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    return (uint32_t)q8_code<FORM>(x.x, s) | (uint32_t)q8_code<FORM>(x.y, s) << 8 | (uint32_t)q8_code<FORM>(x.z, s) << 16 |
           (uint32_t)q8_code<FORM>(x.w, s) << 24;
}

// What takes a sum of products of codes and scaled queries to a score: a key's scale times the row's
// `back`.  At most the largest number: a product beyond it would make a NaN of codes and queries that
// cancel to 0.  Sums of 1 and more leave f32 with either; smaller ones are within what 22 bits of
// queries scaled to 2^13 leave open.
__device__ __forceinline__ float q8_score_unit(float scale, float back) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(scale * back), "f"(3.402823466e38f));
    return r;
}

// The number that a code stands for, before its scale.
template <int FORM>
__device__ __forceinline__ float q8_value(uint8_t c) {
    if constexpr (FORM == kFormInt8)
        return (float)(int8_t)c;
    else
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
template <int FORM>
__device__ __forceinline__ float4 q8_values4(uint32_t c, float s) {
    if constexpr (FORM == kFormE4m3) {
        const float2 u = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3)));
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3)));
        return make_float4(u.x * s, u.y * s, v.x * s, v.y * s);
    }
    return make_float4(q8_value<FORM>((uint8_t)c) * s, q8_value<FORM>((uint8_t)(c >> 8)) * s,
                       q8_value<FORM>((uint8_t)(c >> 16)) * s, q8_value<FORM>((uint8_t)(c >> 24)) * s);
}

}  // namespace vtmu
