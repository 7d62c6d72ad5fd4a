// The normed rotating append's entry point; kernel and launch in pa_rope.cuh.
#include "pa_rope.cuh"

extern "C" pa_status pa_norm_rope_and_cache(void* q_out, void* k_out, const void* q, int64_t q_stride, const void* k,
                                            int64_t k_stride, const void* v, int64_t v_stride, const float* q_weight,
                                            const float* k_weight, float eps, const int32_t* positions,
                                            const float* cos_sin, int32_t max_position, int32_t rot_dim,
                                            int32_t interleaved, void* k_pool, void* v_pool, const int64_t* slot_mapping,
                                            int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t block_size, int32_t num_blocks, pa_dtype in_dtype,
                                            pa_dtype pool_dtype, float k_scale, float v_scale, int32_t* dev_status,
                                            void* stream) {
    if (!std::isfinite(eps) || eps < 0.f) return PA_ERR_INVALID_ARG;
    if (num_tokens > 0) {
        if (!k_weight || (num_q_heads > 0 && !q_weight) || (reinterpret_cast<uintptr_t>(k_weight) & 3u) ||
            (reinterpret_cast<uintptr_t>(q_weight) & 3u) || !pa::aligned16(k_out))
            return PA_ERR_INVALID_ARG;
        // keys in place must be laid out as k_out is
        if (k_out && k == k_out && k_stride != (int64_t)num_kv_heads * head_dim) return PA_ERR_INVALID_ARG;
    }
    return pa::rope_call<true>({q_out, q, q_stride, k, k_stride, v, v_stride, positions, cos_sin, max_position, rot_dim,
                                interleaved, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads, num_kv_heads,
                                head_dim, block_size, num_blocks, in_dtype, pool_dtype, k_scale, v_scale, dev_status,
                                stream, q_weight, k_weight, k_out, eps});
}
