// The rotating append's entry point; kernel and launch in pa_rope.cuh.
#include "pa_rope.cuh"

extern "C" pa_status pa_rope_and_cache(void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                       const void* v, int64_t v_stride, const int32_t* positions, const float* cos_sin,
                                       int32_t max_position, int32_t rot_dim, int32_t interleaved, void* k_pool,
                                       void* v_pool, const int64_t* slot_mapping, int32_t num_tokens,
                                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                       int32_t num_blocks, pa_dtype in_dtype, pa_dtype pool_dtype, float k_scale,
                                       float v_scale, int32_t* dev_status, void* stream) {
    return pa::rope_call<pa::PlainRope>({q_out, q, q_stride, k, k_stride, v, v_stride, positions, cos_sin, max_position, rot_dim,
                                 interleaved, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads, num_kv_heads,
                                 head_dim, block_size, num_blocks, in_dtype, pool_dtype, k_scale, v_scale, dev_status,
                                 stream, nullptr, nullptr, nullptr, 0.f});
}
