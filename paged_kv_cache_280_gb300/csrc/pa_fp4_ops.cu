// 4-bit pools: the quantising append and the unpacking of whole blocks (format and arithmetic in
// pa_fp4.cuh).  Both are bound by HBM: the append reads its rows once and writes 9/16 byte per
// element, the unpacking does the reverse.  A thread takes one group of 16 elements, so a scale is
// found and applied without leaving its registers.
#include <cmath>

#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// Token i, slot s = slots[i]: block s / BS, row s % BS of every KV head's record.
template <typename T, int D>
__global__ void __launch_bounds__(256) reshape_and_cache_fp4_kernel(const T* k_new, const T* v_new, uint8_t* k_pool,
                                                                    uint8_t* v_pool, const int64_t* __restrict__ slots,
                                                                    int32_t num_tokens, int32_t num_kv_heads,
                                                                    int32_t block_size, int64_t pool_slots, float k_scale,
                                                                    float v_scale, int32_t* status) {
    pdl_launch_dependents();
    constexpr int U = D / kFp4Group;
    const int64_t total = (int64_t)num_tokens * num_kv_heads * U;
    for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int u = (int)(idx & (U - 1));
        const uint32_t row = (uint32_t)(idx / U);  // < 2^31 (checked on the host)
        const int tok = (int)(row / (uint32_t)num_kv_heads), h = (int)(row - (uint32_t)tok * (uint32_t)num_kv_heads);
        const int64_t slot = __ldg(slots + tok);
        if (slot < 0) continue;
        if (slot >= pool_slots) {
            if (h == 0 && u == 0) flag_status(status, PA_DEV_BAD_SLOT);
            continue;
        }
        const int64_t blk = slot / block_size, off = slot - blk * block_size;
        const int64_t rec = (blk * num_kv_heads + h) * (int64_t)block_size * fp4_row_bytes(D);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const T* src = (kv ? v_new : k_new) + (int64_t)row * D + kFp4Group * u;
            const float scale = kv ? v_scale : k_scale;
            float y[16];
            load8(src, y);
            load8(src + 8, y + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(y[i], scale);
            bool has_nan;
            const float amax = fp4_amax<16>(y, has_nan);
            float s;
            const uint8_t sb = fp4_scale(amax, has_nan, s);
            uint8_t* dst = (kv ? v_pool : k_pool) + rec;
            *reinterpret_cast<uint2*>(dst + off * (D / 2) + 8 * u) = make_uint2(fp4_codes8(y, s), fp4_codes8(y + 8, s));
            dst[block_size * (D / 2) + off * U + u] = sb;
        }
    }
}

// out[i] = the values of block blocks[i], every KV head, row and element, in T.
template <typename T, int D>
__global__ void __launch_bounds__(256) unpack_blocks_fp4_kernel(const uint8_t* k_pool, const uint8_t* v_pool,
                                                                const int32_t* __restrict__ blocks, int64_t num, T* k_out,
                                                                T* v_out, int32_t num_kv_heads, int32_t block_size,
                                                                int32_t num_blocks, float k_scale, float v_scale,
                                                                int32_t* status) {
    pdl_launch_dependents();
    constexpr int U = D / kFp4Group;
    const int per_block = num_kv_heads * block_size * U;  // < 2^31 (checked on the host)
    const int64_t total = num * per_block;
    for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
         idx += (int64_t)gridDim.x * blockDim.x) {
        const int64_t i = idx / per_block;
        const int within = (int)(idx - i * per_block);
        const int u = within & (U - 1), r = within / U;
        const int h = r / block_size, off = r - h * block_size;
        const int32_t blk = __ldg(blocks + i);
        if (blk < 0 || blk >= num_blocks) {
            if (within == 0) flag_status(status, PA_DEV_BAD_BLOCK_ID);
            continue;
        }
        const int64_t rec = ((int64_t)blk * num_kv_heads + h) * block_size * fp4_row_bytes(D);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* src = (kv ? v_pool : k_pool) + rec;
            const float scale = kv ? v_scale : k_scale;
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + off * (D / 2) + 8 * u));
            const float s = e4m3_to_float(__ldg(src + block_size * (D / 2) + off * U + u));
            float x[16];
            fp4_values8(w.x, s, x);
            fp4_values8(w.y, s, x + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(x[e], scale);
            T* dst = (kv ? v_out : k_out) + idx * kFp4Group;
            store8(dst, x);
            store8(dst + 8, x + 8);
        }
    }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

pa_status fp4_shape_check(int32_t n, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                          pa_dtype dtype, float k_scale, float v_scale) {
    if (n < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32)) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

int grid_for(int64_t threads) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    const int64_t want = (threads + 255) / 256;
    return (int)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_reshape_and_cache_fp4(const void* k_new, const void* v_new, void* k_pool, void* v_pool,
                                              const int64_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                              pa_dtype in_dtype, float k_scale, float v_scale, int32_t* dev_status,
                                              void* stream) {
    using namespace pa;
    const pa_status st = fp4_shape_check(num_tokens, num_kv_heads, head_dim, block_size, num_blocks, in_dtype, k_scale, v_scale);
    if (st != PA_OK) return st;
    if ((int64_t)num_tokens * num_kv_heads >= INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k_new || !v_new || !k_pool || !v_pool || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    const int grid = grid_for((int64_t)num_tokens * num_kv_heads * (head_dim / kFp4Group));
    if (grid <= 0) return PA_ERR_CUDA;
    const int64_t pool_slots = (int64_t)num_blocks * block_size;
    auto go = [&](auto kernel, auto elem) {
        using T = decltype(elem);
        kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const T*>(k_new), static_cast<const T*>(v_new), static_cast<uint8_t*>(k_pool),
            static_cast<uint8_t*>(v_pool), slot_mapping, num_tokens, num_kv_heads, block_size, pool_slots, k_scale, v_scale,
            dev_status);
    };
    if (in_dtype == PA_BF16)
        head_dim == 128 ? go(&reshape_and_cache_fp4_kernel<__nv_bfloat16, 128>, __nv_bfloat16{})
                        : go(&reshape_and_cache_fp4_kernel<__nv_bfloat16, 64>, __nv_bfloat16{});
    else
        head_dim == 128 ? go(&reshape_and_cache_fp4_kernel<float, 128>, 0.f)
                        : go(&reshape_and_cache_fp4_kernel<float, 64>, 0.f);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

extern "C" pa_status pa_unpack_blocks_fp4(const void* k_pool, const void* v_pool, const int32_t* blocks, int32_t num,
                                          void* k_out, void* v_out, int32_t num_kv_heads, int32_t head_dim,
                                          int32_t block_size, int32_t num_blocks, pa_dtype out_dtype, float k_scale,
                                          float v_scale, int32_t* dev_status, void* stream) {
    using namespace pa;
    const pa_status st = fp4_shape_check(num, num_kv_heads, head_dim, block_size, num_blocks, out_dtype, k_scale, v_scale);
    if (st != PA_OK) return st;
    const int64_t per_block = (int64_t)num_kv_heads * block_size * (head_dim / kFp4Group);
    if (per_block >= INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num == 0) return PA_OK;
    if (!k_pool || !v_pool || !blocks || !k_out || !v_out) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out) ||
        (reinterpret_cast<uintptr_t>(blocks) & 3u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    const int grid = grid_for(num * per_block);
    if (grid <= 0) return PA_ERR_CUDA;
    auto go = [&](auto kernel, auto elem) {
        using T = decltype(elem);
        kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
            static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool), blocks, (int64_t)num,
            static_cast<T*>(k_out), static_cast<T*>(v_out), num_kv_heads, block_size, num_blocks, k_scale, v_scale,
            dev_status);
    };
    if (out_dtype == PA_BF16)
        head_dim == 128 ? go(&unpack_blocks_fp4_kernel<__nv_bfloat16, 128>, __nv_bfloat16{})
                        : go(&unpack_blocks_fp4_kernel<__nv_bfloat16, 64>, __nv_bfloat16{});
    else
        head_dim == 128 ? go(&unpack_blocks_fp4_kernel<float, 128>, 0.f) : go(&unpack_blocks_fp4_kernel<float, 64>, 0.f);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
