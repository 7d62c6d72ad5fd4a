// Causal attention of several query rows per sequence over packed keys and values or quantised pools: the simple form,
// one warp per (token, query head), a key at a time with an online softmax in fp32.
#pragma once

#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

enum AttnSource { kAttnPacked = 0, kAttnFp8 = 1, kAttnFp4 = 2 };

struct AttnParams {
    void* out;
    const uint16_t *q, *k, *v;                // q (and packed k, v): bf16
    int64_t q_stride, k_stride, v_stride;     // elements from one token to the next
    const uint8_t *k_pool, *v_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;                  // null: packed
    const int32_t* cu_q_lens;
    int32_t* status;
    int32_t max_blocks_per_seq, num_seqs, num_q_heads, num_kv_heads, num_blocks, num_q_tokens, max_q_len, bs_shift;
    float scale_log2, out_scale;
};

template <int SRC, int D>
__device__ __forceinline__ void attn_row(const AttnParams& p, bool value, int b, int c0, int t, int g, int lane, float* x) {
    constexpr int E = D / 32;
    if constexpr (SRC == kAttnPacked) {
        const uint16_t* row = (value ? p.v : p.k) + (int64_t)(c0 + t) * (value ? p.v_stride : p.k_stride) + g * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = __uint_as_float((uint32_t)row[e] << 16);
    } else {
        const int bs = 1 << p.bs_shift, off = t & (bs - 1);
        int blk = p.block_tables[(int64_t)b * p.max_blocks_per_seq + (t >> p.bs_shift)];
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) flag_status(p.status, PA_DEV_BAD_BLOCK_ID);
            blk = 0;
        }
        const int64_t head = (int64_t)blk * p.num_kv_heads + g;
        if constexpr (SRC == kAttnFp8) {
            const uint8_t* row = (value ? p.v_pool : p.k_pool) + ((head << p.bs_shift) + off) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = e4m3_to_float(row[e]);
        } else {
            const uint8_t* rec = (value ? p.v_pool : p.k_pool) + head * (int64_t)(fp4_row_bytes(D) << p.bs_shift);
            const float s = e4m3_to_float(rec[((D / 2) << p.bs_shift) + off * (D / 16) + lane * E / 16]);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const __half2 c = __half2(__nv_cvt_fp4x2_to_halfraw2(rec[off * (D / 2) + (lane * E + e) / 2], __NV_E2M1));
                x[e] = __low2float(c) * s, x[e + 1] = __high2float(c) * s;
            }
        }
    }
}

template <int SRC, int D>
__global__ void __launch_bounds__(256) attn_kernel(const AttnParams p) {
    constexpr int E = D / 32;
    const int b = blockIdx.y, i = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = p.cu_q_lens[b], n = p.cu_q_lens[b + 1] - c0;
    const int len = SRC == kAttnPacked ? n : p.seq_lens[b];
    if (n == 0) return;
    if (n < 0 || n > len || n > p.max_q_len || c0 < 0 || (int64_t)c0 + n > p.num_q_tokens ||
        (SRC != kAttnPacked && (int64_t)len > ((int64_t)p.max_blocks_per_seq << p.bs_shift))) {
        if (i == 0 && threadIdx.x == 0) flag_status(p.status, PA_DEV_BAD_SEQ_LEN);
        return;
    }
    if (i >= n) return;
    const int G = p.num_q_heads / p.num_kv_heads, pos = len - n + i;
    for (int h = warp; h < p.num_q_heads; h += 8) {
        float q[E], o[E], m = -INFINITY, l = 0.f;
        for (int e = 0; e < E; ++e) {
            q[e] = __uint_as_float((uint32_t)p.q[(int64_t)(c0 + i) * p.q_stride + h * D + lane * E + e] << 16);
            o[e] = 0.f;
        }
        for (int t = 0; t <= pos; ++t) {
            float x[E], s = 0.f;
            attn_row<SRC, D>(p, false, b, c0, t, h / G, lane, x);
            for (int e = 0; e < E; ++e) s += q[e] * x[e];
            for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            s *= p.scale_log2;
            const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
            m = mn, l = l * f + w;
            attn_row<SRC, D>(p, true, b, c0, t, h / G, lane, x);
            for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * x[e];
        }
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(c0 + i) * p.num_q_heads + h) * D + lane * E;
        for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16(o[e] / l * p.out_scale);
    }
}

template <int SRC, int D>
pa_status launch_attn(const AttnParams& p, cudaStream_t st) {
    attn_kernel<SRC, D><<<dim3(p.max_q_len, p.num_seqs), 256, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

bool aligned_to(const void* ptr, unsigned bytes) { return (reinterpret_cast<uintptr_t>(ptr) & (bytes - 1)) == 0; }

}  // namespace
}  // namespace pa
