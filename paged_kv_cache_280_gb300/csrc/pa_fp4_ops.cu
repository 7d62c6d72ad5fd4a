// 4-bit pools: the quantising append and the unpacking of whole blocks (format and arithmetic in
// pa_fp4.cuh).  Both are bound by HBM: the append reads its rows once and writes 9/16 byte per
// element, the unpacking does the reverse.  A thread takes one group of 16 elements, so a scale is
// found and applied without leaving its registers.
#include <cmath>

#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// Token i, slot s = slots[i]: block s / BS, row s % BS of every KV head's record.  A thread takes one group of K
// (blockIdx.y = 0) or of V per turn; a warp's 32 groups are consecutive in the input, and the warp has
// copied those of its next turns ahead into shared memory: the arithmetic (about 200 instructions a group) costs
// nearly as much as HBM takes, so neither may wait for the other.
// Measured, 16383 tokens of 8 heads of 128 in bf16 (86 MB): 17.4 us, 4.9 TB/s.  Steps on the way there: rows loaded
// when their turn comes 22 us, copied two turns ahead 19.5, slots fetched a turn ahead 18.2 -> 17.4; four tokens of a
// head to a warp, which makes whole lines of codes, 27.  Twice the tokens take 32.1 us, fp32 input of 8192 tokens
// 13.9 us (5.5 TB/s): 3 us of each are a launch's ramp and end.  256 tokens of 32 heads take 2.8 us, all ramp.
constexpr int kAppendAhead = 2;
constexpr int kAppendCtas = 4;  // per SM; with 3, 4, 5 and 6: 18.2, 17.4, 19.0, 20.3 us; 256 tokens 3.0, 2.8, 3.2, 3.7
template <typename T, int D>
__global__ void __launch_bounds__(256, kAppendCtas) reshape_and_cache_fp4_kernel(const T* k_new, const T* v_new, uint8_t* k_pool,
                                                                    uint8_t* v_pool, const int64_t* slots, uint32_t total, const FastDiv heads, int32_t bs_shift,
                                                                    int64_t pool_slots, const Divisor kd, const Divisor vd,
                                                                    int32_t* status) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();  // in this order: see rope_and_cache_kernel
    constexpr int U = D / kFp4Group;                     // groups of a row
    constexpr int kGroup = kFp4Group * (int)sizeof(T);   // bytes of a group
    constexpr int kTurn = 32 * kGroup;                   // bytes of a warp's turn
    __shared__ __align__(16) uint8_t ahead[8 * kAppendAhead * kTurn];
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(ahead) + (threadIdx.x >> 5) * kAppendAhead * kTurn;
    const bool is_v = blockIdx.y != 0;
    const uint8_t* in = reinterpret_cast<const uint8_t*>(is_v ? v_new : k_new);
    const uint32_t stride = gridDim.x * 256;
    auto fetch = [&](uint32_t base, int turn) {  // groups base .. base + 31
#pragma unroll
        for (int i = 0; i < kGroup / 16; ++i) {
            const uint32_t chunk = 32 * i + lane;  // 16 bytes each
            if (base + chunk / (kGroup / 16) < total)
                copy_ahead16(ring + turn * kTurn + chunk * 16, in + (size_t)base * kGroup + chunk * 16);
        }
        copies_commit();
    };
    uint32_t base = blockIdx.x * 256 + (threadIdx.x & ~31u);
#pragma unroll
    for (int i = 0; i < kAppendAhead; ++i) fetch(base + i * stride, i);
    const Divisor d = is_v ? vd : kd;
    auto slot_of = [&](uint32_t idx) -> int64_t { return idx < total ? slots[heads.div(idx / U)] : -1; };
    int64_t next = slot_of(base + lane);  // of the turn to come: fetched a turn ahead
    int turn = 0;
    for (; base < total; base += stride) {
        const uint32_t idx = base + lane, u = idx & (U - 1), row = idx / U;
        const uint32_t h = row - heads.div(row) * heads.d;
        const int64_t slot = next;
        next = slot_of(idx + stride);
        copies_wait<kAppendAhead - 1>();
        __syncwarp();  // the other lanes' copies too
        float x[16];
        const uint32_t src = ring + turn * kTurn + lane * kGroup;
        take8<T>(src, 16, x);
        take8<T>(src + kGroup / 2, 16, x + 8);
        __syncwarp();  // read by every lane: the space may be copied into
        fetch(base + kAppendAhead * stride, turn);
        if (++turn == kAppendAhead) turn = 0;
        if (slot < 0) continue;
        if (slot >= pool_slots) {
            if (h == 0 && u == 0) flag_status(status, PA_DEV_BAD_SLOT);
            continue;
        }
        const Fp4Scale f = fp4_scale(amax_nan<16>(x), d);
        uint8_t* rec = (is_v ? v_pool : k_pool) + ((slot >> bs_shift) * heads.d + h) * (int64_t)(fp4_row_bytes(D) << bs_shift);
        const uint32_t off = (uint32_t)slot & ((1u << bs_shift) - 1);
        *reinterpret_cast<uint2*>(rec + off * (D / 2) + 8 * u) = make_uint2(fp4_codes8(x, d, f), fp4_codes8(x + 8, d, f));
        rec[((D / 2) << bs_shift) + off * U + u] = f.byte;
    }
}

// 16 elements to 32-byte-aligned memory in one store (two for fp32): a warp's store covers whole lines.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float* x) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void store16(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 8 * i), "f"(x[8 * i]), "f"(x[8 * i + 1]),
                     "f"(x[8 * i + 2]), "f"(x[8 * i + 3]), "f"(x[8 * i + 4]), "f"(x[8 * i + 5]), "f"(x[8 * i + 6]), "f"(x[8 * i + 7])
                     : "memory");
}

// out[i] = the values of block blocks[i], every KV head, row and element, in T.  A thread takes the same group
// of K and of V, kUnpackPer times, so that four record loads are in flight before the first conversion; a CTA's
// groups are consecutive.  WIDE: the outputs are 32-byte aligned, and a warp's store instruction covers whole lines
// (with two 16-byte stores it covers half of each, and every line reaches L2 twice).
// Measured, 8192 blocks of 16 tokens, 8 heads of 128, to bf16 (688 MB): 103 us, 6.7 TB/s (0.98 of the measured copy
// rate); before the wide stores and pairs of groups 154 us.  To fp32 0.98 as well.  A CTA's 512 places belong to one
// block: with 2 KV heads of 128 or one in 32-token blocks 0.98, with one in 16-token blocks 0.91, with one of 64 0.68.
constexpr int kUnpackPer = 2;
template <typename T, int D, int BS, bool WIDE>
__global__ void __launch_bounds__(256) unpack_blocks_fp4_kernel(const uint8_t* k_pool, const uint8_t* v_pool,
                                                                const int32_t* blocks, uint32_t cta_per_block,
                                                                T* k_out, T* v_out, int32_t num_kv_heads, int32_t num_blocks,
                                                                float k_scale, float v_scale, int32_t* status) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();  // in this order: see rope_and_cache_kernel
    constexpr int U = D / kFp4Group;
    constexpr int kRec = BS * fp4_row_bytes(D);
    const uint32_t i = blockIdx.x / cta_per_block, part = blockIdx.x - i * cta_per_block;
    const int32_t blk = blocks[i];
    if (blk < 0 || blk >= num_blocks) {
        if (part == 0 && threadIdx.x == 0) flag_status(status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const uint32_t per_block = (uint32_t)num_kv_heads * BS * U;  // groups of a block
    uint2 w[kUnpackPer][2];
    uint32_t sb[kUnpackPer][2];
#pragma unroll
    for (int t = 0; t < kUnpackPer; ++t) {
        const uint32_t g = (part * kUnpackPer + t) * 256 + threadIdx.x;
        if (g >= per_block) break;
        const uint32_t h = g / (BS * U), r = g % (BS * U);  // r = row * U + group: the order of the codes and of the scales
        const size_t rec = ((size_t)blk * num_kv_heads + h) * kRec;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t* src = (kv ? v_pool : k_pool) + rec;
            w[t][kv] = *reinterpret_cast<const uint2*>(src + 8 * r);
            sb[t][kv] = src[BS * (D / 2) + r];
        }
    }
#pragma unroll
    for (int t = 0; t < kUnpackPer; ++t) {
        const uint32_t g = (part * kUnpackPer + t) * 256 + threadIdx.x;
        if (g >= per_block) break;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint32_t s = f16x2_low_twice(e4m3x2_to_f16x2(sb[t][kv]));
            const float scale = kv ? v_scale : k_scale;
            float x[16];
            fp4_values8(w[t][kv].x, s, scale, x);
            fp4_values8(w[t][kv].y, s, scale, x + 8);
            T* dst = (kv ? v_out : k_out) + ((size_t)i * per_block + g) * kFp4Group;
            if constexpr (WIDE) {
                store16(dst, x);
            } else {
                store8(dst, x);
                store8(dst + 8, x + 8);
            }
        }
    }
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }
bool aligned32(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 31u) == 0; }

pa_status fp4_shape_check(int32_t n, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                          pa_dtype dtype, float k_scale, float v_scale) {
    if (n < 0 || num_kv_heads <= 0 || num_blocks <= 0) return PA_ERR_INVALID_ARG;
    if (dtype != PA_F32 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32)) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f)) return PA_ERR_INVALID_ARG;
    return PA_OK;
}

struct UnpackArgs {
    const uint8_t *k_pool, *v_pool;
    const int32_t* blocks;
    void *k_out, *v_out;
    int32_t num_kv_heads, num_blocks;
    float k_scale, v_scale;
    int32_t* status;
    unsigned grid, cta_per_block;
    bool wide;
};

template <typename T, int D, int BS>
void launch_unpack(const UnpackArgs& a, cudaStream_t st) {
    auto* kernel = a.wide ? &unpack_blocks_fp4_kernel<T, D, BS, true> : &unpack_blocks_fp4_kernel<T, D, BS, false>;
    launch_dependent(kernel, dim3(a.grid), 256, 0, st, a.k_pool, a.v_pool, a.blocks, a.cta_per_block, static_cast<T*>(a.k_out),
                     static_cast<T*>(a.v_out), a.num_kv_heads, a.num_blocks, a.k_scale, a.v_scale, a.status);
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
    const int64_t total = (int64_t)num_tokens * num_kv_heads * (head_dim / kFp4Group);
    if (total >= INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!k_new || !v_new || !k_pool || !v_pool || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return PA_ERR_CUDA;
    // K and V each: as many CTAs as half the SMs' room for them, or as there is work for
    const int64_t want = (total + 255) / 256, room = (int64_t)sms * kAppendCtas / 2;
    const dim3 grid((unsigned)(want < room ? want : room), 2);
    const int64_t pool_slots = (int64_t)num_blocks * block_size;
    auto go = [&](auto kernel, auto elem) {
        using T = decltype(elem);
        launch_dependent(kernel, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(k_new),
                         static_cast<const T*>(v_new), static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool),
                         slot_mapping, (uint32_t)total, fast_div(num_kv_heads), block_size == 16 ? 4 : 5, pool_slots,
                         divisor(k_scale), divisor(v_scale), dev_status);
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
    const int64_t cta_per_block = (per_block + 256 * kUnpackPer - 1) / (256 * kUnpackPer);
    if (per_block >= INT32_MAX || cta_per_block * num >= INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (num == 0) return PA_OK;
    if (!k_pool || !v_pool || !blocks || !k_out || !v_out) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out) ||
        (reinterpret_cast<uintptr_t>(blocks) & 3u) || (reinterpret_cast<uintptr_t>(dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    const UnpackArgs a{static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool), blocks, k_out, v_out,
                       num_kv_heads, num_blocks, k_scale, v_scale, dev_status, (unsigned)(cta_per_block * num),
                       (unsigned)cta_per_block, aligned32(k_out) && aligned32(v_out)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool b16 = block_size == 16, d128 = head_dim == 128;
    if (out_dtype == PA_BF16)
        d128 ? (b16 ? launch_unpack<__nv_bfloat16, 128, 16>(a, s) : launch_unpack<__nv_bfloat16, 128, 32>(a, s))
             : (b16 ? launch_unpack<__nv_bfloat16, 64, 16>(a, s) : launch_unpack<__nv_bfloat16, 64, 32>(a, s));
    else
        d128 ? (b16 ? launch_unpack<float, 128, 16>(a, s) : launch_unpack<float, 128, 32>(a, s))
             : (b16 ? launch_unpack<float, 64, 16>(a, s) : launch_unpack<float, 64, 32>(a, s));
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
