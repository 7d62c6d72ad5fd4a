// The 4-bit pool format (PA_FP4_E2M1) as the kernels see it.
//
// A row of D elements is D / 16 groups of 16.  Group values are code * s * pool_scale: code one of
// the E2M1 values 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, s the group's E4M3 scale, pool_scale one
// fp32 per pool.  The record of one (block, KV head), BS * (D / 2 + D / 16) bytes, holds the codes of
// its BS token rows and then their scale bytes, both token-major: 9/16 byte per element, and both
// parts of a block and head in one contiguous copy (a multiple of 64 bytes for every shape).
//
// code * s needs at most 6 significant bits (2 of the code, 4 of the scale) and lies in
// {0} u [2^-10, 2688], so it is exact in f16 (and fp32): the readers round nothing but the product
// with the pool scale.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kFp4Group = 16;            // elements per E4M3 scale
constexpr uint8_t kFp4NanScale = 0x7f;   // E4M3 NaN: the whole group reads as NaN

constexpr int fp4_row_bytes(int d) { return d / 2 + d / kFp4Group; }

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// The scale byte of a group whose largest |x / pool_scale| is amax, and the scale's value.  amax / 6
// puts the largest element on the largest code; a group with a NaN gets the NaN scale.
__device__ __forceinline__ uint8_t fp4_scale(float amax, bool has_nan, float& s) {
    const uint8_t b = has_nan ? kFp4NanScale : (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f), __NV_SATFINITE, __NV_E4M3);
    s = e4m3_to_float(b);
    return b;
}

// Eight codes of y[0..7] = x / pool_scale under scale value s, element i in bits 4 i .. 4 i + 3:
// E2M1 of fp32(y / s), nearest even, saturated at 6.  A group whose scale rounds to zero, or is NaN,
// has all codes zero.
__device__ __forceinline__ uint32_t fp4_codes8(const float* y, float s) {
    uint32_t w = 0;
    if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = make_float2(__fdiv_rn(y[2 * i], s), __fdiv_rn(y[2 * i + 1], s));
            w |= (uint32_t)__nv_cvt_float2_to_fp4x2(z, __NV_E2M1, cudaRoundNearest) << (8 * i);
        }
    }
    return w;
}

// max |y[i]| of N values; has_nan when one is a NaN.
template <int N>
__device__ __forceinline__ float fp4_amax(const float* y, bool& has_nan) {
    float a = 0.f;
    has_nan = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a = fmaxf(a, fabsf(y[i]));
        has_nan |= y[i] != y[i];
    }
    return a;
}

// The values (without the pool scale) of the eight codes of w, as fp32.
__device__ __forceinline__ void fp4_values8(uint32_t w, float s, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w >> (8 * i)), __NV_E2M1));
        x[2 * i] = __low2float(h) * s;
        x[2 * i + 1] = __high2float(h) * s;
    }
}

// Eight elements of a row as fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z), x[5] = bf16_hi(r.z), x[6] = bf16_lo(r.w), x[7] = bf16_hi(r.w);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
// Eight fp32 values rounded to the element type and stored.
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                              pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace pa
