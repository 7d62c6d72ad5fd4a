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

#include <cmath>

#include "pa_device.cuh"

namespace pa {

constexpr int kFp4Group = 16;            // elements per E4M3 scale
constexpr uint8_t kFp4NanScale = 0x7f;   // E4M3 NaN: the whole group reads as NaN

constexpr int fp4_row_bytes(int d) { return d / 2 + d / kFp4Group; }

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// ---- fp32 pairs (one instruction for two elements) -----------------------------------------------
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
    uint64_t x, y, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    uint64_t x, y, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    uint64_t x, y, z, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}

// ---- correctly rounded quotients of many elements by one divisor ----------------------------------
// With r the correctly rounded reciprocal of b, q = x r is within 1.5 units in the last place of x / b, and
// q - (q b - x) r, rounded, is x / b correctly rounded (the step is Markstein's, 1990, whose theorem asks for a q
// within one unit).  Take x and b in [1, 2).  For x >= b, q is within one unit and q b - x is exact; for x < b it
// may need 25 bits and lose its last one, 2^-47.  With r's error, 2^-25, times the remainder, what is rounded last
// is within 2^-46 of x / b (2^-47 for x >= b).  So the result could be wrong only where x / b is that near
// to the middle of two floats: x 2^25 - M b (x 2^24 - M b for x >= b) a multiple of 2^-23 below 8, M odd.  All
// such pairs, and those with x next to 1, to 2 and to b, have been computed: none is wrong.  This needs no term to
// leave the normal range: kQuotientMax bounds |x| and b's range (its reciprocal is in range with it).
// Below, where a quotient or a remainder is tiny, the result may be off by a unit of the smallest number; the
// callers round what is so small to zero.  A zero keeps its sign.  For b a power of two q is x / b.
constexpr float kQuotientMax = 1.15292150e18f;  // 2^60

struct Divisor {  // of a launch: b, its reciprocal, whether both are in [2^-60, 2^60], and whether b = 2^n
    float b, r;
    bool in_range, pow2;
};
inline Divisor divisor(float b) {
    int e;
    return Divisor{b, 1.f / b, b <= kQuotientMax && b >= 1.f / kQuotientMax, std::frexp(b, &e) == 0.5f};
}

__device__ __forceinline__ float quotient(float x, float b, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(q, b, -x), -r, q);
}
template <int N>
__device__ __forceinline__ void quotients(const float* x, float b, float r, float* y) {
    const float2 rr = make_float2(r, r), nr = make_float2(-r, -r), bb = make_float2(b, b);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 q = mul_f32x2(make_float2(x[i], x[i + 1]), rr);
        const float2 d = fma_f32x2(fma_f32x2(q, bb, make_float2(-x[i], -x[i + 1])), nr, q);
        y[i] = d.x, y[i + 1] = d.y;
    }
}
template <int N>
__device__ __forceinline__ void quotients(const float* x, const Divisor& d, float* y) {
    if (d.pow2) {
        const float2 rr = make_float2(d.r, d.r);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 q = mul_f32x2(make_float2(x[i], x[i + 1]), rr);
            y[i] = q.x, y[i + 1] = q.y;
        }
    } else {
        quotients<N>(x, d.b, d.r, y);
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // the larger, or NaN if either is
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// max |x[i]| of N (even) values, NaN if one is.
template <int N>
__device__ __forceinline__ float amax_nan(const float* x) {
    float a = max_nan(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
    for (int i = 2; i < N; i += 2)
        asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(a) : "f"(fabsf(x[i])), "f"(fabsf(x[i + 1])));
    return a;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x / b for a b > 0 with the reciprocal r + t (r at most 1 / b, t = (1 - b r) r >= 0): within 2^-41 before its one
// rounding.  Enough where no quotient lies that close to a value that matters (see fp4_codes8).  A zero keeps its
// sign, since t has none.
template <int N>
__device__ __forceinline__ void near_quotients(const float* x, float r, float t, float* y) {
    const float2 rr = make_float2(r, r), tt = make_float2(t, t);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const float2 v = make_float2(x[i], x[i + 1]), d = fma_f32x2(v, rr, mul_f32x2(v, tt));
        y[i] = d.x, y[i + 1] = d.y;
    }
}

// ---- quantisation ---------------------------------------------------------------------------------
// A group's scale from amax, its largest |x| (NaN if it holds one): the byte, and the value and its
// reciprocal for fp4_codes8.  Division is monotonic, so max |x / b| is amax / b; a sixth of it puts the
// largest element on the largest code.
struct Fp4Scale {
    float s, r, t;  // s, and its reciprocal as r + t
    uint8_t byte;
    bool plain;  // fp4_codes8 may use quotients()
};
__device__ __forceinline__ Fp4Scale fp4_scale(float amax, const Divisor& d) {
    Fp4Scale f;
    f.plain = d.in_range && amax <= kQuotientMax;
    if (f.plain) {
        f.byte = (uint8_t)__nv_cvt_float_to_fp8(quotient(quotient(amax, d.b, d.r), 6.f, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
    } else if (amax != amax) {
        f.byte = kFp4NanScale;
    } else {
        f.byte = (uint8_t)__nv_cvt_float_to_fp8(__fdiv_rn(__fdiv_rn(amax, d.b), 6.f), __NV_SATFINITE, __NV_E4M3);
    }
    f.s = e4m3_to_float(f.byte);
    // The hardware's reciprocal is within 2^-23 of 1 / s; 2^-22 less is below it, by less than 2^-21.  Then
    // 1 - s r is exact (s has 4 significant bits), and r + t is within (2^-21)^2 and t's rounding of 1 / s.
    f.r = f.s > 0.f ? rcp_approx(f.s) * (1.f - 0x1p-22f) : 0.f;  // 0: every code zero
    f.t = __fmaf_rn(-f.s, f.r, 1.f) * f.r;
    return f;
}

// Eight codes of x under a group's scale, element i in bits 4 i .. 4 i + 3: E2M1 of fp32(fp32(x / b) / s),
// nearest even, saturated at 6, with x's sign.  All zero where the scale is zero or NaN.
// The inner quotient y is exact to its rounding.  The outer one only has to fall on the right side of, or on, the
// codes' midpoints m: m s is an fp32 number of at most 7 significant bits, so y is m s itself, and y / s comes
// out as m, or differs from it by 2^-24 of it or more.
__device__ __forceinline__ uint32_t fp4_codes8(const float* x, const Divisor& d, const Fp4Scale& f) {
    float y[8];
    if (f.plain) {
        quotients<8>(x, d, y);
        near_quotients<8>(y, f.r, f.t, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = f.s > 0.f ? __fdiv_rn(__fdiv_rn(x[i], d.b), f.s) : 0.f;
    }
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return f.r > 0.f ? w : 0u;
}

// Two E4M3 bytes (low byte first) to an f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
    uint32_t d;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(b));
    return d;
}
// The eight codes of w to four f16 pairs: byte i to r[i], the byte's low code in the low half.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t f16x2_low_twice(uint32_t v) { return __byte_perm(v, 0, 0x1010); }
__device__ __forceinline__ uint32_t f16x2_high_twice(uint32_t v) { return __byte_perm(v, 0, 0x3232); }

// The values of the eight codes of w times the pool scale, as fp32: code * s in f16 (exact; s a pair of the
// group's scale), then one fp32 rounding.
__device__ __forceinline__ void fp4_values8(uint32_t w, uint32_t s, float pool_scale, float* x) {
    uint32_t r[4];
    e2m1x8_to_f16x2(w, r);
    const float2 p = make_float2(pool_scale, pool_scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = mul_f16x2(r[i], s);
        const float2 y = mul_f32x2(make_float2(f16_lo(v), f16_hi(v)), p);
        x[2 * i] = y.x, x[2 * i + 1] = y.y;
    }
}

// n / d for n < 2^31 and a launch's d >= 1, as a multiplication: q = (high word of n m, plus n) >> s with
// s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1 (Granlund and Montgomery 1994).
struct FastDiv {
    uint32_t d, m, s;
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return FastDiv{d, (uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}

// ---- rows copied ahead -----------------------------------------------------------------------------
// Copies from global to shared memory, 16 bytes a thread, some turns of a loop ahead: the bytes in flight then
// need no registers.  CA: through L1, for copies of half a sector each, so that the other half is found there.
template <bool CA = false>
__device__ __forceinline__ void copy_ahead16(uint32_t dst, const void* src) {
    if constexpr (CA)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups of this thread's copies have landed
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// Eight elements of T in shared memory as fp32: 16 bytes, or for fp32 two times 16, `step` bytes apart.
template <typename T>
__device__ __forceinline__ void take8(uint32_t src, uint32_t step, float* x) {
    const uint4 a = lds16(src);
    if constexpr (sizeof(T) == 2) {
        x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
        x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
    } else {
        const uint4 b = lds16(src + step);
        x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
        x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y), x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    }
}

// Eight elements of a row as fp32.
__device__ __forceinline__ void widen8(const uint4& r, float* x) {
    x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z), x[5] = bf16_hi(r.z), x[6] = bf16_lo(r.w), x[7] = bf16_hi(r.w);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) { widen8(*reinterpret_cast<const uint4*>(p), x); }
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
