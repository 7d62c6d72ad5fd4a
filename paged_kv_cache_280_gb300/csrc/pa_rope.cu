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
// Work: a row is one head of one token; a thread takes 16 elements of it, the two 8-element halves of
// eight pairs, so that both elements of a pair meet in its registers with 16-byte loads and stores
// in either pairing, and in-place queries are read and written by the same thread.
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
    float k_scale, v_scale;
    int32_t* status;
    int32_t num_tokens, num_q_heads, num_kv_heads, block_size, max_position, rot_dim, interleaved;
};

__device__ __forceinline__ uint2 fp8_codes8(const float* x, float scale) {
    uint32_t w[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        w[half] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[half] |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[4 * half + e], scale), __NV_SATFINITE, __NV_E4M3) << (8 * e);
    }
    return make_uint2(w[0], w[1]);
}

template <typename T, int POOL, int D>
__global__ void __launch_bounds__(256) rope_and_cache_kernel(const RopeParams p) {
    pdl_launch_dependents();  // a decode that follows may start its prologue (it reads nothing written here)
    constexpr int U = D / 16;  // threads per row
    const int H = p.num_q_heads + 2 * p.num_kv_heads;
    const int64_t total = (int64_t)p.num_tokens * H * U;
    const int half = p.rot_dim / 2;
    // every thread of a warp takes the same number of turns: the 4-bit pool's groups meet in shuffles
    for (int64_t base = (int64_t)blockIdx.x * blockDim.x; base < total; base += (int64_t)gridDim.x * blockDim.x) {
        const int64_t idx = base + threadIdx.x;
        const bool in_range = idx < total;
        const int u = (int)(idx & (U - 1));
        const uint32_t row = in_range ? (uint32_t)(idx / U) : 0u;  // < 2^31 (checked on the host)
        const int tok = (int)(row / (uint32_t)H), h = (int)(row - (uint32_t)tok * (uint32_t)H);
        const int64_t slot = p.slots[tok];
        bool ok = in_range && slot >= 0;
        int pos = 0;
        if (ok) {
            pos = p.positions[tok];
            const bool bad_slot = slot >= p.pool_slots, bad_pos = pos < 0 || pos >= p.max_position;
            if (bad_slot || bad_pos) {
                ok = false;
                if (h == 0 && u == 0)
                    flag_status(p.status, (bad_slot ? PA_DEV_BAD_SLOT : 0) | (bad_pos ? PA_DEV_BAD_POSITION : 0));
            }
        }
        const bool is_q = h < p.num_q_heads, is_v = h >= p.num_q_heads + p.num_kv_heads;
        const bool turned = !is_v && 16 * u < p.rot_dim;
        const bool apart = turned && !p.interleaved;  // the halves of this unit lie rot_dim / 2 apart
        const int e0 = apart ? 8 * u : 16 * u, e1 = apart ? half + 8 * u : 16 * u + 8;
        float a[8], b[8];
        if (ok) {
            const T* src = is_q   ? static_cast<const T*>(p.q) + tok * p.q_stride + h * D
                           : is_v ? static_cast<const T*>(p.v) + tok * p.v_stride + (h - p.num_q_heads - p.num_kv_heads) * D
                                  : static_cast<const T*>(p.k) + tok * p.k_stride + (h - p.num_q_heads) * D;
            load8(src + e0, a);
            load8(src + e1, b);
            if (turned) {
                float c[8], s[8];
                const float* cs = p.cos_sin + (int64_t)pos * p.rot_dim + 8 * u;
                load8(cs, c);
                load8(cs + half, s);
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float& x = i < 4 ? a[2 * (i & 3)] : b[2 * (i & 3)];
                        float& y = i < 4 ? a[2 * (i & 3) + 1] : b[2 * (i & 3) + 1];
                        const float nx = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
                        y = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
                        x = nx;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float na = __fsub_rn(__fmul_rn(a[i], c[i]), __fmul_rn(b[i], s[i]));
                        b[i] = __fadd_rn(__fmul_rn(b[i], c[i]), __fmul_rn(a[i], s[i]));
                        a[i] = na;
                    }
                }
            }
            if (is_q) {
                T* dst = static_cast<T*>(p.q_out) + ((int64_t)tok * p.num_q_heads + h) * D;
                store8(dst + e0, a);
                store8(dst + e1, b);
            }
        }
        const bool append = ok && !is_q;
        const int kvh = is_v ? h - p.num_q_heads - p.num_kv_heads : h - p.num_q_heads;
        const int64_t blk = slot / p.block_size, off = slot - blk * p.block_size;
        uint8_t* pool = is_v ? p.v_pool : p.k_pool;
        const float scale = is_v ? p.v_scale : p.k_scale;
        if constexpr (POOL == kPoolFp4) {
            float y0[8], y1[8];
            float m0 = 0.f, m1 = 0.f;
            bool n0 = false, n1 = false;
            if (append) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y0[i] = __fdiv_rn(a[i], scale);
                    y1[i] = __fdiv_rn(b[i], scale);
                }
                m0 = fp4_amax<8>(y0, n0);
                m1 = fp4_amax<8>(y1, n1);
            }
            // a unit whose halves lie apart shares both its groups with its neighbour (rot_dim is a
            // multiple of 32); any other unit is one group
            const float o0 = __shfl_xor_sync(0xffffffffu, m0, 1), o1 = __shfl_xor_sync(0xffffffffu, m1, 1);
            const int nans = (n0 ? 1 : 0) | (n1 ? 2 : 0);
            const int onans = __shfl_xor_sync(0xffffffffu, nans, 1);
            if (append) {
                const float g0 = apart ? fmaxf(m0, o0) : fmaxf(m0, m1), g1 = apart ? fmaxf(m1, o1) : g0;
                const bool h0 = apart ? ((nans | onans) & 1) != 0 : nans != 0;
                const bool h1 = apart ? ((nans | onans) & 2) != 0 : h0;
                float s0, s1;
                const uint8_t b0 = fp4_scale(g0, h0, s0), b1 = fp4_scale(g1, h1, s1);
                uint8_t* rec = pool + (blk * p.num_kv_heads + kvh) * (int64_t)p.block_size * fp4_row_bytes(D);
                uint8_t* codes = rec + off * (D / 2);
                uint8_t* scales = rec + p.block_size * (D / 2) + off * (D / kFp4Group);
                *reinterpret_cast<uint32_t*>(codes + e0 / 2) = fp4_codes8(y0, s0);
                *reinterpret_cast<uint32_t*>(codes + e1 / 2) = fp4_codes8(y1, s1);
                if (!apart || (u & 1) == 0) {
                    scales[e0 / kFp4Group] = b0;
                    if (apart) scales[e1 / kFp4Group] = b1;
                }
            }
        } else {
            if (append) {
                const int64_t r = (blk * p.num_kv_heads + kvh) * p.block_size + off;  // the slot's row in the pool
                if constexpr (POOL == kPoolFp8) {
                    *reinterpret_cast<uint2*>(pool + r * D + e0) = fp8_codes8(a, scale);
                    *reinterpret_cast<uint2*>(pool + r * D + e1) = fp8_codes8(b, scale);
                } else {
                    T* dst = reinterpret_cast<T*>(pool) + r * D;
                    store8(dst + e0, a);
                    store8(dst + e1, b);
                }
            }
        }
    }
}

template <typename T, int D>
void launch_rope(const RopeParams& p, pa_dtype pool, int grid, cudaStream_t st) {
    if (pool == PA_FP4_E2M1)
        rope_and_cache_kernel<T, kPoolFp4, D><<<grid, 256, 0, st>>>(p);
    else if (pool == PA_FP8_E4M3)
        rope_and_cache_kernel<T, kPoolFp8, D><<<grid, 256, 0, st>>>(p);
    else
        rope_and_cache_kernel<T, kPoolSame, D><<<grid, 256, 0, st>>>(p);
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
    if (heads * num_tokens >= INT32_MAX) return PA_ERR_UNSUPPORTED;
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
    p.k_scale = k_scale, p.v_scale = v_scale;
    p.status = dev_status;
    p.num_tokens = num_tokens, p.num_q_heads = num_q_heads, p.num_kv_heads = num_kv_heads;
    p.block_size = block_size, p.max_position = max_position, p.rot_dim = rot_dim, p.interleaved = interleaved;
    const int64_t want = (heads * num_tokens * (head_dim / 16) + 255) / 256;
    const int grid = (int)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (in_dtype == PA_BF16)
        head_dim == 128 ? launch_rope<__nv_bfloat16, 128>(p, pool_dtype, grid, st)
                        : launch_rope<__nv_bfloat16, 64>(p, pool_dtype, grid, st);
    else
        head_dim == 128 ? launch_rope<float, 128>(p, pool_dtype, grid, st) : launch_rope<float, 64>(p, pool_dtype, grid, st);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
