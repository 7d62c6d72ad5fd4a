// Chunk attention over FP8 and 4-bit pools: entry points and checks; the kernel in pa_attn.cuh.
#include <cmath>
#include <cstring>

#include "pa_attn.cuh"

namespace pa {
namespace {

// The status head, then, from the next 256-byte boundary on, the cut unit that begins in each CTA and two slots per CTA for
// pieces of cut units: a maximum and a sum per row, and the rows.
struct PrefillWorkspace {
    size_t ml, o, total;
    int tiles;
};
PrefillWorkspace prefill_workspace(int max_q_len, int group, int head_dim, int sms) {
    PrefillWorkspace w;
    w.tiles = max_q_len > kAtRows / group ? 2 : 1;
    w.ml = ((size_t)sms * sizeof(int4) + 255) & ~(size_t)255;
    const size_t rows = (size_t)2 * sms * w.tiles * kAtRows;
    w.o = w.ml + rows * sizeof(float2);
    w.total = 2 * kStatusHeadBytes + w.o + rows * head_dim * sizeof(float);
    return w;
}

pa_status prefill_quant(void* out, const void* q, const void* k_pool, const void* v_pool, float k_scale, float v_scale,
                        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                        const int32_t* cu_q_lens, int32_t num_seqs, int32_t num_q_tokens, int32_t max_q_len,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int32_t num_blocks, float scale, void* workspace, size_t workspace_bytes, bool fp4, void* stream) {
    if (num_seqs <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || max_q_len < 0 ||
        num_q_tokens < 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || !std::isfinite(scale) || !(scale > 0.f) ||
        !std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f))
        return PA_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > 8 || (head_dim != 128 && !(fp4 && head_dim == 64)) ||
        (block_size != 16 && block_size != 32) || num_seqs > 65535 || num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    if (max_q_len == 0 || num_q_tokens == 0) return PA_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !cu_q_lens || !workspace) return PA_ERR_INVALID_ARG;
    if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(k_pool, 16) || !aligned_to(v_pool, 16) ||
        !aligned_to(workspace, 16) || !aligned_to(block_tables, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_q_lens, 4))
        return PA_ERR_INVALID_ARG;
    const float scale_log2 = scale * k_scale * 1.4426950408889634f;
    if (!std::isfinite(scale_log2) || !(scale_log2 > 0.f)) return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return PA_ERR_CUDA;
    const int group = num_q_heads / num_kv_heads;
    const PrefillWorkspace ws = prefill_workspace(max_q_len, group, head_dim, sms);
    if (workspace_bytes < ws.total) return PA_ERR_WORKSPACE_TOO_SMALL;
    AttnParams p = {};
    p.out = out;
    p.q = static_cast<const uint16_t*>(q);
    p.k_pool = static_cast<const uint8_t*>(k_pool), p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.block_tables = block_tables, p.seq_lens = seq_lens, p.cu_q_lens = cu_q_lens;
    p.status = static_cast<int32_t*>(workspace);
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + kStatusHeadBytes + 255) & ~(uintptr_t)255);
    p.cuts = reinterpret_cast<int4*>(base);
    p.part_ml = reinterpret_cast<float2*>(base + ws.ml), p.part_o = reinterpret_cast<float*>(base + ws.o);
    p.part_tiles = ws.tiles;
    p.max_blocks_per_seq = max_blocks_per_seq, p.num_seqs = num_seqs, p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads, p.num_blocks = num_blocks, p.num_q_tokens = num_q_tokens, p.max_q_len = max_q_len;
    p.bs_shift = block_size == 16 ? 4 : 5;
    const int64_t held = (int64_t)max_blocks_per_seq * block_size;
    p.max_len = (int32_t)(held < kAttnMaxLen ? held : kAttnMaxLen);
    p.group = group, p.tile_tokens = kAtRows / group;
    p.group_inverse = (65536u + p.group - 1) / p.group;
    p.wait_limit_ns = (int32_t)wait_limit_ns();
    p.out_align32 = aligned_to(out, 32) ? 1 : 0;
    // the same product as a number in [1, 2] and its power of two (its factors may lie near fp32's ends, and so may the rows')
    int e_scale, e_pool, e_product;
    const float product = std::frexp(scale, &e_scale) * std::frexp(k_scale, &e_pool) * 1.4426950408889634f;
    p.scale_log2 = 2.f * std::frexp(product, &e_product);
    p.scale_exp = e_scale + e_pool + e_product - 1;
    p.out_scale = v_scale;
    CUtensorMap none;  // not read: the codes come by bulk copies
    memset(&none, 0, sizeof none);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!fp4) return launch_attn<kAttnFp8, 128>(p, dev, sms, none, none, none, st);
    return head_dim == 128 ? launch_attn<kAttnFp4, 128>(p, dev, sms, none, none, none, st)
                           : launch_attn<kAttnFp4, 64>(p, dev, sms, none, none, none, st);
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_prefill_workspace_bytes(int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
                                                int32_t head_dim, size_t* bytes_out) {
    if (!bytes_out || max_q_len < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || head_dim <= 0)
        return PA_ERR_INVALID_ARG;
    if (num_q_heads / num_kv_heads > 8) return PA_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    if (!pa::current_device(&dev, &sms)) return PA_ERR_CUDA;
    *bytes_out = pa::prefill_workspace(max_q_len, num_q_heads / num_kv_heads, head_dim, sms).total;
    return PA_OK;
}

extern "C" pa_status pa_prefill_attention_fp8(void* out, const void* q, const void* k_pool, const void* v_pool,
                                              float k_scale, float v_scale, const int32_t* block_tables,
                                              int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                              const int32_t* cu_q_lens, int32_t num_seqs, int32_t num_q_tokens,
                                              int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    return pa::prefill_quant(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                             num_seqs, num_q_tokens, max_q_len, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                             scale, workspace, workspace_bytes, false, stream);
}

extern "C" pa_status pa_prefill_attention_fp4(void* out, const void* q, const void* k_pool, const void* v_pool,
                                              float k_scale, float v_scale, const int32_t* block_tables,
                                              int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                              const int32_t* cu_q_lens, int32_t num_seqs, int32_t num_q_tokens,
                                              int32_t max_q_len, int32_t num_q_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t block_size, int32_t num_blocks, float scale,
                                              void* workspace, size_t workspace_bytes, void* stream) {
    return pa::prefill_quant(out, q, k_pool, v_pool, k_scale, v_scale, block_tables, max_blocks_per_seq, seq_lens, cu_q_lens,
                             num_seqs, num_q_tokens, max_q_len, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                             scale, workspace, workspace_bytes, true, stream);
}
