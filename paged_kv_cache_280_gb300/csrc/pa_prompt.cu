// Attention over whole prompts, packed one behind the other: entry point and checks; the kernel in pa_attn.cuh.
#include <cmath>

#include "pa_attn.cuh"

namespace pa {
namespace {

// Largest distance between tokens of a strided q, k or v, in elements: a tensor map holds strides below 2^40 bytes.
constexpr int64_t kMaxRowStride = (int64_t)1 << 38;

// The TMA map of bf16 rows [tokens][heads][head_dim] with `stride` elements from one token to the next, viewed as
// (head_dim, heads, tokens): one box = 64 elements x box_heads x box_tokens with the 128-byte swizzle.
bool rows_map(CUtensorMap* map, const void* rows, int64_t tokens, int heads, int head_dim, int64_t stride, int box_heads,
              int box_tokens) {
    const auto encode = tensor_map_encoder();
    if (!encode) return false;
    cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(rows), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_prompt_attention(void* out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* v, int64_t v_stride, const int32_t* cu_lens, int32_t num_seqs,
                                         int32_t num_tokens, int32_t max_len, int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, float scale, pa_dtype dtype, int32_t* dev_status,
                                         void* stream) {
    using namespace pa;
    if (dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || max_len < 0 ||
        num_tokens < 0 || !std::isfinite(scale) || !(scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > 8 || (head_dim != 64 && head_dim != 128) || num_seqs > 65535 || num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)num_q_heads * head_dim || k_stride < (int64_t)num_kv_heads * head_dim ||
        v_stride < (int64_t)num_kv_heads * head_dim || q_stride % 8 || k_stride % 8 || v_stride % 8)
        return PA_ERR_INVALID_ARG;
    if (q_stride > kMaxRowStride || k_stride > kMaxRowStride || v_stride > kMaxRowStride) return PA_ERR_UNSUPPORTED;
    if (max_len == 0 || num_tokens == 0) return PA_OK;
    if (!out || !q || !k || !v || !cu_lens) return PA_ERR_INVALID_ARG;
    if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(cu_lens, 4) ||
        !aligned_to(dev_status, 4))
        return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return PA_ERR_CUDA;
    AttnParams p = {};
    p.out = out;
    p.cu_q_lens = cu_lens, p.status = dev_status;
    p.num_seqs = num_seqs, p.num_q_heads = num_q_heads, p.num_kv_heads = num_kv_heads;
    p.num_q_tokens = num_tokens, p.max_q_len = max_len < num_tokens ? max_len : num_tokens;
    p.group = num_q_heads / num_kv_heads, p.tile_tokens = kAtRows / p.group;
    p.group_inverse = (65536u + p.group - 1) / p.group;
    p.wait_limit_ns = (int32_t)wait_limit_ns();
    p.out_align32 = aligned_to(out, 32) ? 1 : 0;
    p.scale_log2 = scale * 1.4426950408889634f, p.out_scale = 1.f;
    if (!std::isfinite(p.scale_log2) || !(p.scale_log2 > 0.f)) return PA_ERR_INVALID_ARG;
    CUtensorMap tq, tk, tv;
    if (!rows_map(&tq, q, num_tokens, num_q_heads, head_dim, q_stride, p.group, p.tile_tokens) ||
        !rows_map(&tk, k, num_tokens, num_kv_heads, head_dim, k_stride, 1, kAttnKeys) ||
        !rows_map(&tv, v, num_tokens, num_kv_heads, head_dim, v_stride, 1, kAttnKeys))
        return PA_ERR_CUDA;
    // a CTA per unit where there are fewer than SMs
    const int64_t units = most_packed_units(num_seqs, num_tokens, p.max_q_len, num_kv_heads, p.tile_tokens);
    const int grid = (int)(units < sms ? units : sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch_attn<kAttnPacked, 128>(p, dev, grid, tq, tk, tv, st)
                           : launch_attn<kAttnPacked, 64>(p, dev, grid, tq, tk, tv, st);
}
