// Softmax state of a decode warp over a 4-bit pool (format: pa_fp4.cuh), on the tensor cores
// (mma.sync m16n8k16, f16 operands, fp32 sums).
//
// The bound.  A token row of one KV head is 9/16 D bytes of K and the same of V (144 bytes at D = 128),
// and every code has to become an f16 in registers: at the measured HBM rate an SM receives a token
// row pair every 6 cycles, so the consumer has about 25 issue slots for its 2 D elements, 8 per lane.
// The fragments are laid out so that an element costs one half of a conversion and one half of a
// multiplication by its group's scale, which is exact in f16, and nothing is moved between lanes:
//  - S^T = K q^T, 16 tokens x 8 heads.  Lane (g, c) = (lane / 4, lane % 4) reads D / 4 consecutive
//    dims of its two token rows at once (16 bytes at D = 128: two scale groups).  The order of a dot
//    product's terms is free, so k-step j takes each lane's dims 4 j .. 4 j + 3 and q's fragments
//    hold the same dims.
//  - O^T = V^T P^T, 16 dims x 8 heads.  Lane (g, c) reads the D / 8 dims from D / 8 g of its four
//    tokens (at D = 128 one scale group).  A nibble merge of two tokens' words pairs the tokens of
//    each dim, which a conversion turns into the f16 pair of an A operand; m16 block i holds dims
//    2 i (row g) and 2 i + 1 (row g + 8) of each lane's run, which the stores undo.
//  - Tokens: the 16 slots of a step are permuted so that the row reads of S spread over the
//    shared-memory banks and those of V over half of them (slot_token below).
//  - The row sums l come from one more MMA, whose A operand is all ones: they are sums of the rounded
//    weights that P V uses, and need no reduction over lanes.
//  - The sums are fp32, and a tensor core cuts each product at about 2^-23 of the sum that it joins: n tokens of one
//    warp's piece are off by at most n 2^-23 of their sum, and O and l alike.
// As built a token row costs 16.9 warp instructions at D = 128 (70.7 million for 4 sequences of 131,072 tokens and 8 KV
// heads), of the 25 slots above; on 96 sequences of 32 heads the issue slots are 63 % busy.
// Slots past the sequence's end may hold any bits: their scores become -inf, and their V rows get
// scale 0 (codes are always finite), so neither reaches the output.
#pragma once

#include "pa_fp4.cuh"

namespace pa {

__device__ __forceinline__ float ex2_approx(float x) {  // 2^x, 2^-inf = 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// N consecutive 32-bit words of shared memory (N = 1, 2 or 4, naturally aligned).
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

template <int D, int BS>
struct Fp4State {
    static constexpr int MT = D / 16;       // m16 blocks of O^T, and 16-dim k-steps of S
    static constexpr int KW = D / 32;       // words of a lane's part of a K row (D / 4 dims)
    static constexpr int VW = D / 64;       // words of a lane's part of a V row (D / 8 dims)
    static constexpr int kScalesOff = BS * (D / 2);  // the tile's scale bytes
    uint32_t qb[MT][2];  // B fragments of q^T per k-step, rows scaled by a power of two
    float sc[2];         // score scale (base 2, > 0) of heads 2c and 2c + 1, the power of two undone
    float m[2];          // reference of heads 2c, 2c + 1: a score before its scale, the same in every g
    float l[4];          // running sums: [0], [1] of heads 2c, 2c + 1 (the same in every g; [2], [3] repeat them)
    float o[MT][4];

    // token of slot r (0..7) of a step; slot r + 8 holds token + 8
    __device__ static __forceinline__ int slot_token(int r) { return 4 * (r & 1) + ((r >> 1) ^ (r & 1)); }
    // token of the i-th (0..3) of the slots 2c, 2c + 1, 2c + 8, 2c + 9 of lane c: slot_token in c's terms
    __device__ static __forceinline__ int lane_token(int c, int i) { return 4 * i + (c ^ (i & 1)); }

    __device__ __forceinline__ void reset() {
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = l[2] = l[3] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }

    // f16 holds a bf16 value exactly while it is neither above 65504 nor far below 2^-14, so each row is
    // scaled by the power of two that brings its largest element to [1, 2): a smaller element loses
    // less than 2^-25 of that one, and any bf16 magnitudes are in range.  A negative score scale turns the
    // rows' signs, so that sc is positive; it is kept so (and finite) where it would round to 0.
    // rows: q[b][h * G] in global memory.
    __device__ __forceinline__ void load_q(const __nv_bfloat16* rows, int G, int lane, float scale_log2) {
        const int g = lane >> 2, c = lane & 3;
        float x[D / 4];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            if (g < G) {
                load8(rows + g * D + c * (D / 4) + 8 * i, x + 8 * i);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[8 * i + e] = 0.f;
            }
        }
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) a = fmaxf(a, fabsf(x[i]));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const int e = min(max((int)(__float_as_uint(a) >> 23), 1), 253);
        const float f = copysignf(__uint_as_float((uint32_t)(254 - e) << 23), scale_log2);
        const float inv = __uint_as_float((uint32_t)e << 23);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            qb[j][0] = pack_f16x2(x[4 * j] * f, x[4 * j + 1] * f);
            qb[j][1] = pack_f16x2(x[4 * j + 2] * f, x[4 * j + 3] * f);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            sc[i] = fminf(fmaxf(fabsf(scale_log2) * __shfl_sync(0xffffffffu, inv, 8 * c + 4 * i), 0x1p-126f), 0x1.fffffep127f);
    }

    // S^T of the 16 tokens from row row0 of the tile at kbase: (slot g, head 2c), (g, 2c + 1),
    // (g + 8, 2c), (g + 8, 2c + 1).
    __device__ __forceinline__ void scores(uint32_t kbase, int row0, int lane, float (&acc)[4]) const {
        const int g = lane >> 2, c = lane & 3;
        const int row = row0 + slot_token(g);
        uint32_t w0[KW], w1[KW];
        lds_words<KW>(kbase + row * (D / 2) + c * (D / 8), w0);
        lds_words<KW>(kbase + (row + 8) * (D / 2) + c * (D / 8), w1);
        const uint32_t sa = kbase + kScalesOff + row * (D / 16) + c * (D / 64);
        uint32_t s0[2], s1[2];  // the lane's scale groups of each row, twice in a pair
        if constexpr (D == 128) {
            const uint32_t p0 = e4m3x2_to_f16x2(lds_u16(sa)), p1 = e4m3x2_to_f16x2(lds_u16(sa + 8 * (D / 16)));
            s0[0] = f16x2_low_twice(p0), s0[1] = f16x2_high_twice(p0);
            s1[0] = f16x2_low_twice(p1), s1[1] = f16x2_high_twice(p1);
        } else {
            s0[0] = s0[1] = f16x2_low_twice(e4m3x2_to_f16x2(lds_u8(sa)));
            s1[0] = s1[1] = f16x2_low_twice(e4m3x2_to_f16x2(lds_u8(sa + 8 * (D / 16))));
        }
        float acc2[4] = {0.f, 0.f, 0.f, 0.f};  // two independent chains over the k-steps
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t x0[4], x1[4];
            e2m1x8_to_f16x2(w0[w], x0);
            e2m1x8_to_f16x2(w1[w], x1);
            const uint32_t k0 = s0[w / 2], k1 = s1[w / 2];  // 16 dims: two words to a group
            mma_f16_16816(acc, mul_f16x2(x0[0], k0), mul_f16x2(x1[0], k1), mul_f16x2(x0[1], k0), mul_f16x2(x1[1], k1),
                          qb[2 * w][0], qb[2 * w][1]);
            mma_f16_16816(acc2, mul_f16x2(x0[2], k0), mul_f16x2(x1[2], k1), mul_f16x2(x0[3], k0), mul_f16x2(x1[3], k1),
                          qb[2 * w + 1][0], qb[2 * w + 1][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += acc2[i];
    }

    // O^T += V^T P^T and l += sum P of the 16 tokens from row row0 of the tile at vbase; MASK: only the
    // first `valid` of them exist.
    template <bool MASK>
    __device__ __forceinline__ void accumulate_pv(uint32_t vbase, int row0, int valid, uint32_t b0, uint32_t b1, int lane) {
        const int g = lane >> 2, c = lane & 3;
        uint32_t v[4][VW], sb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = lane_token(c, i);
            lds_words<VW>(vbase + (row0 + t) * (D / 2) + g * (D / 16), v[i]);
            sb[i] = lds_u8(vbase + kScalesOff + (row0 + t) * (D / 16) + (D == 128 ? g : g >> 1));
            if (MASK && t >= valid) sb[i] = 0;
        }
        const uint32_t s01 = e4m3x2_to_f16x2(sb[0] | (sb[1] << 8)), s23 = e4m3x2_to_f16x2(sb[2] | (sb[3] << 8));
        constexpr uint32_t kOnes = 0x3c003c00u, kLow = 0x0f0f0f0fu;
        mma_f16_16816(l, kOnes, kOnes, kOnes, kOnes, b0, b1);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            uint32_t even01[4], odd01[4], even23[4], odd23[4];
            e2m1x8_to_f16x2((v[0][w] & kLow) | ((v[1][w] & kLow) << 4), even01);
            e2m1x8_to_f16x2(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), odd01);
            e2m1x8_to_f16x2((v[2][w] & kLow) | ((v[3][w] & kLow) << 4), even23);
            e2m1x8_to_f16x2(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), odd23);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_f16_16816(o[4 * w + i], mul_f16x2(even01[i], s01), mul_f16x2(odd01[i], s01), mul_f16x2(even23[i], s23),
                              mul_f16x2(odd23[i], s23), b0, b1);
        }
    }

    // A stage holds 32 tokens, two 16-token steps, with one softmax update.  MASK: only the first `valid`
    // (1 .. 32) of them exist.  Tile t's K is at kb + t * tile bytes, its V at vb + t * tile bytes.
    static constexpr int kTile = BS * fp4_row_bytes(D), kStep1 = BS == 16 ? kTile : 0, kRow1 = BS == 16 ? 0 : 16;

    // The weights of the stage's tokens as P^T B fragments (step 0: pb[0], pb[1]; step 1: pb[2], pb[3]):
    // 2^((x - m) sc + kAbove) of the scores x.  The difference comes before the scale, so the reference's own exponent
    // is kAbove however large the scores are (x sc - m sc, the second rounded, is off by half a unit of m sc: 64 at 2^30).
    // m is a reference, not the exact maximum: it moves (and O and l are rescaled) only when a score
    // passes it by more than 2^(kRaise - kAbove), so that most stages need no reduction over lanes.  The weights
    // then stay at most 2^kRaise, within f16, and the final ratio does not depend on the reference.
    // (The reduction and the rescaling are 9 shuffles and 4 MT + 4 multiplications a stage.)
    // kAbove puts the largest weight near the top of f16: a weight keeps its 11 bits down to 2^-25 of the largest one of
    // its piece, and below is off by at most 2^-36 of it, so that a long tail of small weights is not lost.  A reference
    // that moves after 2^4 costs no more than one that moves after 2^8 (kAbove 7): the same times on 20 batches.
    static constexpr float kRaise = 15.f, kAbove = 11.f;
    template <bool MASK>
    __device__ __forceinline__ void weights(uint32_t kb, int valid, int lane, uint32_t (&pb)[4]) {
        const int g = lane >> 2;
        float x[2][4], y[2][4];  // scores; base-2 exponents of the weights
        scores(kb, 0, lane, x[0]);
        scores(kb + kStep1, kRow1, lane, x[1]);
        auto exponents = [&]() {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {  // a token's two heads
                    const float2 d = add_f32x2(make_float2(x[s][i], x[s][i + 1]), make_float2(-m[0], -m[1]));
                    const float2 e = fma_f32x2(d, make_float2(sc[0], sc[1]), make_float2(kAbove, kAbove));
                    const bool past = MASK && slot_token(g) + 8 * (i >> 1) + 16 * s >= valid;
                    y[s][i] = past ? -INFINITY : e.x, y[s][i + 1] = past ? -INFINITY : e.y;
                }
        };
        exponents();  // +inf while m = -inf: no score has been seen
        const float top = max3(max3(y[0][0], y[0][1], y[0][2]), max3(y[0][3], y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3]));
        if (__any_sync(0xffffffffu, top > kRaise)) {
            float n[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                n[i] = -INFINITY;
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        if (!MASK || slot_token(g) + 8 * r + 16 * s < valid) n[i] = fmaxf(n[i], x[s][2 * r + i]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) n[i] = fmaxf(n[i], __shfl_xor_sync(0xffffffffu, n[i], off));
                n[i] = fmaxf(n[i], m[i]);
            }
            // a head whose scores are all -inf so far keeps its state (nothing is weighed yet)
            const float a0 = n[0] == m[0] ? 1.f : ex2_approx((m[0] - n[0]) * sc[0]);
            const float a1 = n[1] == m[1] ? 1.f : ex2_approx((m[1] - n[1]) * sc[1]);
            l[0] *= a0, l[1] *= a1, l[2] *= a0, l[3] *= a1;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][0] *= a0, o[i][1] *= a1, o[i][2] *= a0, o[i][3] *= a1;
            m[0] = n[0], m[1] = n[1];
            exponents();
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            pb[2 * s] = movmatrix_trans(pack_f16x2(ex2_approx(y[s][0]), ex2_approx(y[s][1])));
            pb[2 * s + 1] = movmatrix_trans(pack_f16x2(ex2_approx(y[s][2]), ex2_approx(y[s][3])));
        }
    }

    // O and l with those weights.
    template <bool MASK>
    __device__ __forceinline__ void accumulate(uint32_t vb, int valid, int lane, const uint32_t (&pb)[4]) {
        accumulate_pv<MASK>(vb, 0, valid, pb[0], pb[1], lane);
        accumulate_pv<MASK>(vb + kStep1, kRow1, valid - 16, pb[2], pb[3], lane);
    }

    // Normalised output rows (o_rows = out[b][h * G]): a lane holds D / 8 consecutive dims of its two heads.
    // The pool scale comes last: divided by l, which may be 2^40, a small one would leave the normal range.
    __device__ __forceinline__ void store_out(__nv_bfloat16* o_rows, int G, int lane, float oscale) const {
        const int g = lane >> 2, h0 = 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (h0 + j < G) {
                const float r = 1.f / l[j];
                __nv_bfloat16* dst = o_rows + (h0 + j) * D + g * (D / 8);
#pragma unroll
                for (int i = 0; i < MT; i += 4)
                    *reinterpret_cast<uint4*>(dst + 2 * i) =
                        make_uint4(pack_bf16x2(o[i][j] * r * oscale, o[i][2 + j] * r * oscale),
                                   pack_bf16x2(o[i + 1][j] * r * oscale, o[i + 1][2 + j] * r * oscale),
                                   pack_bf16x2(o[i + 2][j] * r * oscale, o[i + 2][2 + j] * r * oscale),
                                   pack_bf16x2(o[i + 3][j] * r * oscale, o[i + 3][2 + j] * r * oscale));
            }
        }
    }

    // Unnormalised partial: slot = [G][D] o, then [G] (m, l), m in base 2 (that of weight 1).
    __device__ __forceinline__ void store_partial(float* slot, int G, int lane) const {
        const int g = lane >> 2, h0 = 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (h0 + j < G) {
                float* dst = slot + (h0 + j) * D + g * (D / 8);
#pragma unroll
                for (int i = 0; i < MT; i += 2)
                    *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(o[i][j], o[i][2 + j], o[i + 1][j], o[i + 1][2 + j]);
                if (g == 0) {
                    slot[G * D + 2 * (h0 + j)] = fmaf(m[j], sc[j], -kAbove);
                    slot[G * D + 2 * (h0 + j) + 1] = l[j];
                }
            }
        }
    }
};

}  // namespace pa
