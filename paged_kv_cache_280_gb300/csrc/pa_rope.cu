// Rotating append: queries and keys turned by their positions, keys and values appended to the paged
// pools, in one pass over q, k and v.
//
// Token i at position p, pair j of the first rot_dim elements of a query or key head, (a, b) its two
// elements (j and j + rot_dim / 2, or 2 j and 2 j + 1 when interleaved), c = cos_sin[p][j] and
// s = cos_sin[p][rot_dim / 2 + j]:
//     a' = a c - b s,   b' = b c + a s,
// in fp32 with every product and the sum rounded (no fused multiply-add), so that the same fp32
// expression anywhere gives the same bits, and the same codes in a quantised pool.  The turned key is
// rounded once, to the pool's type.
//
// Bound: HBM.  A call reads q, k, v and the cos / sin rows and writes q_out and the pool rows once.
// Work: a unit is 16 elements of one head of one token, the two 8-element halves of eight pairs, so that
// both elements of a pair meet in one thread's registers with 16-byte loads and stores in either
// pairing, and in-place queries are read and written by the same thread.  A thread takes the same unit of
// HPT heads of a token: their loads are in flight together, and the unit's cos and sin are fetched once.
#include <cmath>

#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

enum RopePool { kPoolSame = 0, kPoolFp8 = 1, kPoolFp4 = 2 };

struct RopeParams {
    void* q_out;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    const int32_t* positions;
    const float* cos_sin;
    const int64_t* slots;
    uint8_t *k_pool, *v_pool;
    int64_t pool_slots;
    Divisor k_scale, v_scale;
    int32_t* status;
    int32_t num_tokens, num_q_heads, num_kv_heads, bs_shift, max_position, rot_dim, interleaved;
    uint32_t head_groups;  // threads' groups of heads per token
};

// E4M3 codes of fp32(x / scale), nearest even, saturated at 448.
__device__ __forceinline__ uint2 fp8_codes8(const float* x, const Divisor& d) {
    float y[8];
    if (d.in_range && amax_nan<8>(x) <= kQuotientMax) {
        quotients<8>(x, d.b, d.r, y);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], d.b);
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const float2 z = make_float2(copysignf(y[e], x[e]), copysignf(y[e + 1], x[e + 1]));
        w[e / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3) << (8 * (e & 2));
    }
    return make_uint2(w[0], w[1]);
}

// Eight elements as loaded: 16 bytes of bf16, or 32 of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void widen(float* x) const { widen8(r, x); }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void widen(float* x) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

template <typename T, int POOL, int D, int HPT>
__global__ void __launch_bounds__(256) rope_and_cache_kernel(const RopeParams p) {
    pdl_launch_dependents();  // a decode that follows may start its prologue (it reads nothing written here)
    constexpr int U = D / 16;  // units per row
    const uint32_t total = (uint32_t)p.num_tokens * p.head_groups * U;  // < 2^31 (checked on the host)
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x;  // every thread of a warp stays: 4-bit groups meet in shuffles
    const bool in_range = idx < total;
    const int u = (int)(idx & (U - 1));
    const uint32_t group = in_range ? idx / U : 0u;
    const uint32_t tok = group / p.head_groups;
    const int h0 = (int)(group - tok * p.head_groups) * HPT, H = p.num_q_heads + 2 * p.num_kv_heads;
    const int half = p.rot_dim / 2;
    const bool rot_unit = 16 * u < p.rot_dim, split_unit = rot_unit && !p.interleaved;
    auto is_q = [&](int h) { return h < p.num_q_heads; };
    auto is_v = [&](int h) { return h >= p.num_q_heads + p.num_kv_heads; };
    // a unit of two halves rot_dim / 2 apart, or of 16 consecutive elements
    auto apart = [&](int h) { return split_unit && !is_v(h); };
    auto e0 = [&](int h) { return apart(h) ? 8 * u : 16 * u; };
    auto e1 = [&](int h) { return apart(h) ? half + 8 * u : 16 * u + 8; };
    // the rows first: they need neither slot nor position
    Raw8<T> ra[HPT], rb[HPT];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = h0 + i;
        if (in_range && h < H) {
            const T* src = is_q(h)   ? static_cast<const T*>(p.q) + tok * p.q_stride + h * D
                           : is_v(h) ? static_cast<const T*>(p.v) + tok * p.v_stride + (h - p.num_q_heads - p.num_kv_heads) * D
                                     : static_cast<const T*>(p.k) + tok * p.k_stride + (h - p.num_q_heads) * D;
            ra[i].load(src + e0(h));
            rb[i].load(src + e1(h));
        }
    }
    const int64_t slot = p.slots[tok];
    bool ok = in_range && slot >= 0;
    int pos = 0;
    if (ok) {
        pos = p.positions[tok];
        const bool bad_slot = slot >= p.pool_slots, bad_pos = pos < 0 || pos >= p.max_position;
        if (bad_slot || bad_pos) {
            ok = false;
            if (h0 == 0 && u == 0)
                flag_status(p.status, (bad_slot ? PA_DEV_BAD_SLOT : 0) | (bad_pos ? PA_DEV_BAD_POSITION : 0));
        }
    }
    float c[8], s[8];
    if (ok && rot_unit && !is_v(h0)) {
        const float* cs = p.cos_sin + (int64_t)pos * p.rot_dim + 8 * u;
        load8(cs, c);
        load8(cs + half, s);
    }
    const uint32_t off = (uint32_t)slot & ((1u << p.bs_shift) - 1);
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        const int h = h0 + i;
        const bool live = ok && h < H;
        float a[8], b[8];
        if (live) {
            ra[i].widen(a);
            rb[i].widen(b);
            if (rot_unit && !is_v(h)) {
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float& x = j < 4 ? a[2 * (j & 3)] : b[2 * (j & 3)];
                        float& y = j < 4 ? a[2 * (j & 3) + 1] : b[2 * (j & 3) + 1];
                        const float nx = __fsub_rn(__fmul_rn(x, c[j]), __fmul_rn(y, s[j]));
                        y = __fadd_rn(__fmul_rn(y, c[j]), __fmul_rn(x, s[j]));
                        x = nx;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float na = __fsub_rn(__fmul_rn(a[j], c[j]), __fmul_rn(b[j], s[j]));
                        b[j] = __fadd_rn(__fmul_rn(b[j], c[j]), __fmul_rn(a[j], s[j]));
                        a[j] = na;
                    }
                }
            }
            if (is_q(h)) {
                T* dst = static_cast<T*>(p.q_out) + ((int64_t)tok * p.num_q_heads + h) * D;
                store8(dst + e0(h), a);
                store8(dst + e1(h), b);
            }
        }
        const bool append = live && !is_q(h);
        const int kvh = is_v(h) ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads;
        uint8_t* pool = is_v(h) ? p.v_pool : p.k_pool;
        const int64_t head = (slot >> p.bs_shift) * p.num_kv_heads + kvh;  // the (block, KV head) in the pool
        if constexpr (POOL == kPoolFp4) {
            // a unit whose halves lie apart shares both its groups with its neighbour (rot_dim is a
            // multiple of 32); any other unit is one group
            float m0 = 0.f, m1 = 0.f;
            if (append) m0 = amax_nan<8>(a), m1 = amax_nan<8>(b);
            const float o0 = __shfl_xor_sync(0xffffffffu, m0, 1), o1 = __shfl_xor_sync(0xffffffffu, m1, 1);
            if (append) {
                const Divisor d = is_v(h) ? p.v_scale : p.k_scale;
                const bool ap = apart(h);
                const Fp4Scale f0 = fp4_scale(max_nan(m0, ap ? o0 : m1), d);
                Fp4Scale f1 = f0;
                if (ap) f1 = fp4_scale(max_nan(m1, o1), d);
                uint8_t* rec = pool + head * (int64_t)(fp4_row_bytes(D) << p.bs_shift);
                uint8_t* codes = rec + off * (D / 2);
                uint8_t* scales = rec + ((D / 2) << p.bs_shift) + off * (D / kFp4Group);
                const uint32_t w0 = fp4_codes8(a, d, f0), w1 = fp4_codes8(b, d, f1);
                if (ap) {
                    *reinterpret_cast<uint32_t*>(codes + 4 * u) = w0;
                    *reinterpret_cast<uint32_t*>(codes + half / 2 + 4 * u) = w1;
                    if ((u & 1) == 0) {
                        scales[u / 2] = f0.byte;
                        scales[half / kFp4Group + u / 2] = f1.byte;
                    }
                } else {
                    *reinterpret_cast<uint2*>(codes + 8 * u) = make_uint2(w0, w1);
                    scales[u] = f0.byte;
                }
            }
        } else if (append) {
            const int64_t r = (head << p.bs_shift) + off;  // the slot's row in the pool
            if constexpr (POOL == kPoolFp8) {
                const Divisor d = is_v(h) ? p.v_scale : p.k_scale;
                *reinterpret_cast<uint2*>(pool + r * D + e0(h)) = fp8_codes8(a, d);
                *reinterpret_cast<uint2*>(pool + r * D + e1(h)) = fp8_codes8(b, d);
            } else {
                T* dst = reinterpret_cast<T*>(pool) + r * D;
                store8(dst + e0(h), a);
                store8(dst + e1(h), b);
            }
        }
    }
}

template <typename T, int POOL, int D>
void launch_hpt(RopeParams& p, int sms, cudaStream_t st) {
    // Four heads to a thread once that still fills the SMs twice over (latency is short by then against the
    // stream); one to a thread for a decode batch.
    constexpr int kMany = sizeof(T) == 4 ? 2 : 4;
    const int64_t heads = (int64_t)p.num_q_heads + 2 * p.num_kv_heads, units = p.num_tokens * heads * (D / 16);
    const int hpt = units / kMany >= (int64_t)sms * 2048 * 2 ? kMany : 1;
    p.head_groups = (uint32_t)((heads + hpt - 1) / hpt);
    const unsigned grid = (unsigned)(((int64_t)p.num_tokens * p.head_groups * (D / 16) + 255) / 256);
    if (hpt == 1)
        rope_and_cache_kernel<T, POOL, D, 1><<<grid, 256, 0, st>>>(p);
    else
        rope_and_cache_kernel<T, POOL, D, kMany><<<grid, 256, 0, st>>>(p);
}

template <typename T, int D>
void launch_rope(RopeParams& p, pa_dtype pool, int sms, cudaStream_t st) {
    if (pool == PA_FP4_E2M1)
        launch_hpt<T, kPoolFp4, D>(p, sms, st);
    else if (pool == PA_FP8_E4M3)
        launch_hpt<T, kPoolFp8, D>(p, sms, st);
    else
        launch_hpt<T, kPoolSame, D>(p, sms, st);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_rope_and_cache(void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                                       int32_t max_position, int32_t rot_dim, int32_t interleaved, void* k_pool,
                                       void* v_pool, const int64_t* slot_mapping, int32_t num_tokens,
                                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int32_t num_blocks, pa_dtype in_dtype, pa_dtype pool_dtype, float k_scale,
                                       float v_scale, int32_t* dev_status, void* stream) {
    using namespace pa;
    if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks <= 0 || max_position <= 0 || rot_dim <= 0 ||
        (interleaved != 0 && interleaved != 1))
        return PA_ERR_INVALID_ARG;
    if (in_dtype != PA_F32 && in_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    const bool quantised = pool_dtype == PA_FP8_E4M3 || pool_dtype == PA_FP4_E2M1;
    if (!quantised && pool_dtype != in_dtype) return PA_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32) ||
        (pool_dtype == PA_FP8_E4M3 && head_dim != 128))
        return PA_ERR_UNSUPPORTED;
    if (rot_dim > head_dim) return PA_ERR_INVALID_ARG;
    if (rot_dim % (pool_dtype == PA_FP4_E2M1 ? 32 : 16)) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f)) return PA_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)num_q_heads + 2 * (int64_t)num_kv_heads;
    if (heads * num_tokens * (head_dim / 16) >= INT32_MAX) return PA_ERR_UNSUPPORTED;
    const int64_t per16 = in_dtype == PA_F32 ? 4 : 8;  // elements in 16 bytes
    if ((num_q_heads > 0 && q_stride < (int64_t)num_q_heads * head_dim) || k_stride < (int64_t)num_kv_heads * head_dim ||
        v_stride < (int64_t)num_kv_heads * head_dim || (num_q_heads > 0 && q_stride % per16) || k_stride % per16 ||
        v_stride % per16)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if ((num_q_heads > 0 && (!q || !q_out)) || !k || !v || !positions || !cos_sin || !k_pool || !v_pool || !slot_mapping)
        return PA_ERR_INVALID_ARG;
    if ((num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) || !aligned16(k) || !aligned16(v) || !aligned16(cos_sin) ||
        !aligned16(k_pool) || !aligned16(v_pool) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    // queries in place must be laid out as q_out is
    if (num_q_heads > 0 && q == q_out && q_stride != (int64_t)num_q_heads * head_dim) return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return PA_ERR_CUDA;
    RopeParams p;
    p.q_out = q_out, p.q = q, p.k = k, p.v = v;
    p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.slots = slot_mapping;
    p.k_pool = static_cast<uint8_t*>(k_pool), p.v_pool = static_cast<uint8_t*>(v_pool);
    p.pool_slots = (int64_t)num_blocks * block_size;
    p.k_scale = divisor(k_scale), p.v_scale = divisor(v_scale);
    p.status = dev_status;
    p.num_tokens = num_tokens, p.num_q_heads = num_q_heads, p.num_kv_heads = num_kv_heads;
    p.bs_shift = block_size == 16 ? 4 : 5, p.max_position = max_position, p.rot_dim = rot_dim, p.interleaved = interleaved;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (in_dtype == PA_BF16)
        head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, pool_dtype, sms, st)
                        : launch_rope<__nv_bfloat16, 64>(p, pool_dtype, sms, st);
    else
        head_dim == 128 ? launch_rope<float, 128>(p, pool_dtype, sms, st) : launch_rope<float, 64>(p, pool_dtype, sms, st);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
