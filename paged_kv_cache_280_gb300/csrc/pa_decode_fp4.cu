// Decode over 4-bit pools with bf16 queries and outputs, on the tensor cores for every group size
// (pa_decode_fp4.cuh has the arithmetic and its bound).
#include "pa_decode.cuh"

namespace pa {

bool decode_variant_fp4(int head_dim, int block_size, int group, DecodeVariant* out) {
    if (head_dim == 128 && block_size == 16) *out = VariantOf<__nv_bfloat16, 128, 16, true, 0, Fp4>::get();
    else if (head_dim == 128 && block_size == 32) *out = VariantOf<__nv_bfloat16, 128, 32, true, 0, Fp4>::get();
    else if (head_dim == 64 && block_size == 16) *out = VariantOf<__nv_bfloat16, 64, 16, true, 0, Fp4>::get();
    else if (head_dim == 64 && block_size == 32) *out = VariantOf<__nv_bfloat16, 64, 32, true, 0, Fp4>::get();
    else return false;
    return true;
}

}  // namespace pa
