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
// Work: a unit is 16 elements of one head of one token in two runs of eight, rot_dim / 2 apart (past rot_dim:
// half of the rest apart): both elements of a pair meet in one thread's registers in either pairing, and
// eight threads' runs are consecutive.  In-place queries are read and written by the same thread.  A thread
// takes a unit per turn and has copied the units of its next turns ahead into shared memory, so that enough
// bytes are in flight whatever the arithmetic (and the quantised pools' registers) cost.
#pragma once

#include <cmath>

#include "pa_fp4.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

enum RopePool { kPoolSame = 0, kPoolFp8 = 1, kPoolFp4 = 2 };

// Measured: 8191 tokens of 64 + 16 heads of 128, bf16 to bf16 (340 MB): 50.9 us, 6.7 TB/s (0.99 of the measured copy
// rate); with the loads of a unit issued when its turn comes 70 us, with only its slot and position fetched then
// 54.6.  4096 fp32 tokens of 32 + 16 heads 34.0 us (0.89), bf16 ones to FP8 pools 18.8 (0.75).  4099 tokens of 32 + 16 heads
// to 4-bit pools 21.4 us (0.63: two groups' codes cost more than HBM takes).  One token: 1.9 us, a launch and one trip
// to memory.
// CTAs per SM: 4 (64 registers); with 5 it spills and is slower, with 3 the 4-bit case takes 23.8 us.
constexpr int kRopeAhead = 2;  // turns that a thread copies ahead

struct RopeParams {
    void* q_out;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
    const int32_t* positions;
    const float* cos_sin;
    const int64_t* slots;
    uint8_t *k_pool, *v_pool;
    int64_t pool_slots;
    Divisor k_scale, v_scale;
    int32_t* status;
    int32_t num_tokens, num_q_heads, num_kv_heads, bs_shift, max_position, rot_dim, interleaved;
    FastDiv heads;  // of a token: queries, keys, values
    // of the normed form: weights fp32 [D] and the turned keys' dense copy (or null)
    const float *q_weight, *k_weight;
    void* k_out;
    float eps;
    FastDiv q_heads, kv_heads;  // of a token: queries; keys and values
};

// E4M3 codes of fp32(x / scale), nearest even, saturated at 448.
__device__ __forceinline__ uint2 fp8_codes8(const float* x, const Divisor& d) {
    float y[8];
    if (d.in_range && amax_nan<8>(x) <= kQuotientMax) {
        quotients<8>(x, d, y);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = __fdiv_rn(x[e], d.b);
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        w[e / 4] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[e], y[e + 1]), __NV_SATFINITE, __NV_E4M3) << (8 * (e & 2));
    }
    return make_uint2(w[0], w[1]);
}

// A unit's 16 elements, two runs of eight at e0 and e1 of a key or value head, to its row of the pool.  Every thread of a
// warp comes here: 4-bit groups meet in shuffles.
template <typename T, int POOL, int D>
__device__ __forceinline__ void append_unit(const RopeParams& p, bool append, bool is_v, int kvh, int64_t slot, int u, int e0, int e1,
                                            const float (&a)[8], const float (&b)[8]) {
    uint8_t* pool = is_v ? p.v_pool : p.k_pool;
    const int64_t head = (slot >> p.bs_shift) * p.num_kv_heads + kvh;  // the (block, KV head) in the pool
    const uint32_t off = (uint32_t)slot & ((1u << p.bs_shift) - 1);
    if constexpr (POOL == kPoolFp4) {
        // a run is half a group of 16, the neighbour's the other half (rot_dim is a multiple of 32)
        float m0 = 0.f, m1 = 0.f;
        if (append) m0 = amax_nan<8>(a), m1 = amax_nan<8>(b);
        const float o0 = __shfl_xor_sync(0xffffffffu, m0, 1), o1 = __shfl_xor_sync(0xffffffffu, m1, 1);
        if (append) {
            const Divisor d = is_v ? p.v_scale : p.k_scale;
            const Fp4Scale f0 = fp4_scale(max_nan(m0, o0), d), f1 = fp4_scale(max_nan(m1, o1), d);
            uint8_t* rec = pool + head * (int64_t)(fp4_row_bytes(D) << p.bs_shift);
            uint8_t* codes = rec + off * (D / 2);
            uint8_t* scales = rec + ((D / 2) << p.bs_shift) + off * (D / kFp4Group);
            *reinterpret_cast<uint32_t*>(codes + e0 / 2) = fp4_codes8(a, d, f0);
            *reinterpret_cast<uint32_t*>(codes + e1 / 2) = fp4_codes8(b, d, f1);
            // of the pair, the even thread writes the first run's scale, the odd one the second's
            scales[((u & 1) ? e1 : e0) / kFp4Group] = (u & 1) ? f1.byte : f0.byte;
        }
    } else if (append) {
        const int64_t r = (head << p.bs_shift) + off;  // the slot's row in the pool
        if constexpr (POOL == kPoolFp8) {
            const Divisor d = is_v ? p.v_scale : p.k_scale;
            *reinterpret_cast<uint2*>(pool + r * D + e0) = fp8_codes8(a, d);
            *reinterpret_cast<uint2*>(pool + r * D + e1) = fp8_codes8(b, d);
        } else {
            T* dst = reinterpret_cast<T*>(pool) + r * D;
            store8(dst + e0, a);
            store8(dst + e1, b);
        }
    }
}

template <typename T, int POOL, int D>
__global__ void __launch_bounds__(256, 4) rope_and_cache_kernel(const RopeParams p) {
    // A decode that follows may start its prologue, which reads nothing written here, but only once what came
    // before this kernel is complete: that may have written the lengths and tables it reads.
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    constexpr int U = D / 16;  // units per row
    constexpr int kParts = (int)sizeof(T) / 2;      // 16-byte parts of a run
    constexpr uint32_t kPart = 256 * 16;            // one part of every thread's run
    constexpr uint32_t kTurn = 2 * kParts * kPart;  // two runs
    __shared__ __align__(16) uint8_t ahead[kRopeAhead * kTurn];
    const uint32_t mine = smem_u32(ahead) + threadIdx.x * 16;
    const int H = p.num_q_heads + 2 * p.num_kv_heads, first_v = p.num_q_heads + p.num_kv_heads, half = p.rot_dim / 2;
    const uint32_t total = (uint32_t)p.num_tokens * (uint32_t)H * U;  // < 2^30 (checked on the host)
    const int u = (int)(threadIdx.x & (U - 1));
    const bool rot_unit = 16 * u < p.rot_dim;
    const int e0 = rot_unit ? 8 * u : 8 * u + half;                            // = rot_dim + 8 (u - rot_dim / 16)
    const int e1 = rot_unit ? 8 * u + half : 8 * u + half + (D - p.rot_dim) / 2;
    const uint32_t first = blockIdx.x * 256u + threadIdx.x, stride = gridDim.x * 256u;
    auto row_of = [&](uint32_t idx, uint32_t& tok, int& h) {
        const uint32_t row = idx / U;
        tok = p.heads.div(row);
        h = (int)(row - tok * p.heads.d);
    };
    auto fetch = [&](uint32_t idx, int turn) {
        if (idx < total) {
            uint32_t tok;
            int h;
            row_of(idx, tok, h);
            const T* src = h < p.num_q_heads ? static_cast<const T*>(p.q) + tok * p.q_stride + h * D
                           : h < first_v     ? static_cast<const T*>(p.k) + tok * p.k_stride + (h - p.num_q_heads) * D
                                             : static_cast<const T*>(p.v) + tok * p.v_stride + (h - first_v) * D;
            const uint32_t dst = mine + turn * kTurn;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                copy_ahead16<kParts == 2>(dst + i * kPart, src + e0 + 4 * i);
                copy_ahead16<kParts == 2>(dst + (kParts + i) * kPart, src + e1 + 4 * i);
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) fetch(first + i * stride, i);
    int turn = 0;
    // The slot and position of the turn to come, fetched a turn ahead, but not for the 4-bit pools, whose arithmetic
    // wants the registers (21.8 us with it on the case above).
    constexpr bool kPlaceAhead = POOL != kPoolFp4;
    int64_t slot_ahead = -1;
    int pos_ahead = 0;
    auto fetch_place = [&](uint32_t tok) { slot_ahead = p.slots[tok], pos_ahead = p.positions[tok]; };
    if constexpr (kPlaceAhead) fetch_place(p.heads.div((first < total ? first : 0u) / U));
    // every thread of a warp takes the same number of turns: 4-bit groups meet in shuffles
    for (uint32_t base = first & ~31u; base < total; base += stride) {
        const uint32_t idx = base + (threadIdx.x & 31u);
        const bool in_range = idx < total;
        uint32_t tok;
        int h;
        row_of(in_range ? idx : 0u, tok, h);
        const bool is_q = h < p.num_q_heads, is_v = h >= first_v;
        if constexpr (!kPlaceAhead) fetch_place(tok);
        const int64_t slot = slot_ahead;
        const int pos = pos_ahead;  // (of a padding token: not looked at)
        if constexpr (kPlaceAhead) fetch_place(p.heads.div((idx + stride < total ? idx + stride : 0u) / U));
        bool ok = in_range && slot >= 0;
        if (ok) {
            const bool bad_slot = slot >= p.pool_slots, bad_pos = pos < 0 || pos >= p.max_position;
            if (bad_slot || bad_pos) {
                ok = false;
                if (h == 0 && u == 0)
                    flag_status(p.status, (bad_slot ? PA_DEV_BAD_SLOT : 0) | (bad_pos ? PA_DEV_BAD_POSITION : 0));
            }
        }
        const bool turned = ok && rot_unit && !is_v;
        float c[8], s[8];
        if (turned) {
            const float* cs = p.cos_sin + (int64_t)pos * p.rot_dim;
            if (p.interleaved) {  // four pairs of each run
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pair = (i ? e1 : e0) / 2;
                    const float4 cv = *reinterpret_cast<const float4*>(cs + pair), sv = *reinterpret_cast<const float4*>(cs + half + pair);
                    c[4 * i] = cv.x, c[4 * i + 1] = cv.y, c[4 * i + 2] = cv.z, c[4 * i + 3] = cv.w;
                    s[4 * i] = sv.x, s[4 * i + 1] = sv.y, s[4 * i + 2] = sv.z, s[4 * i + 3] = sv.w;
                }
            } else {
                load8(cs + e0, c);
                load8(cs + half + e0, s);
            }
        }
        copies_wait<kRopeAhead - 1>();
        float a[8], b[8];
        take8<T>(mine + turn * kTurn, kPart, a);
        take8<T>(mine + turn * kTurn + kParts * kPart, kPart, b);
        fetch(idx + kRopeAhead * stride, turn);
        if (++turn == kRopeAhead) turn = 0;
        if (turned) {
            if (p.interleaved) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float& x = j < 4 ? a[2 * (j & 3)] : b[2 * (j & 3)];
                    float& y = j < 4 ? a[2 * (j & 3) + 1] : b[2 * (j & 3) + 1];
                    const float nx = __fsub_rn(__fmul_rn(x, c[j]), __fmul_rn(y, s[j]));
                    y = __fadd_rn(__fmul_rn(y, c[j]), __fmul_rn(x, s[j]));
                    x = nx;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float na = __fsub_rn(__fmul_rn(a[j], c[j]), __fmul_rn(b[j], s[j]));
                    b[j] = __fadd_rn(__fmul_rn(b[j], c[j]), __fmul_rn(a[j], s[j]));
                    a[j] = na;
                }
            }
        }
        if (ok && is_q) {
            T* dst = static_cast<T*>(p.q_out) + ((int64_t)tok * p.num_q_heads + h) * D;
            store8(dst + e0, a);
            store8(dst + e1, b);
        }
        const bool append = ok && !is_q;
        append_unit<T, POOL, D>(p, append, is_v, is_v ? h - first_v : h - p.num_q_heads, slot, u, e0, e1, a, b);
    }
}

// How a form is launched: its kernel, and its units (of a thread and turn) to a grid.
struct PlainRope {
    template <typename T, int POOL, int D>
    static auto kernel() { return &rope_and_cache_kernel<T, POOL, D>; }
    static constexpr int kThreads = 256;
    static unsigned grid(RopeParams&, int64_t units, int resident) {
        const int64_t want = (units + 255) / 256;
        return (unsigned)(want < resident ? want : resident);
    }
};

template <typename FORM, typename T, int POOL, int D>
bool launch_pool(RopeParams p, int dev, int sms, cudaStream_t st) {
    auto* kernel = FORM::template kernel<T, POOL, D>();
    int occ = 0;
    if (!kernel_occupancy(dev, reinterpret_cast<const void*>(kernel), FORM::kThreads, 0, &occ) || occ <= 0) return false;
    const unsigned grid = FORM::grid(p, (int64_t)p.num_tokens * p.heads.d * (D / 16), sms * occ);
    return launch_dependent(kernel, dim3(grid), FORM::kThreads, 0, st, p) == cudaSuccess;
}

template <typename FORM, typename T, int D>
bool launch_rope(const RopeParams& p, pa_dtype pool, int dev, int sms, cudaStream_t st) {
    return pool == PA_FP4_E2M1   ? launch_pool<FORM, T, kPoolFp4, D>(p, dev, sms, st)
           : pool == PA_FP8_E4M3 ? launch_pool<FORM, T, kPoolFp8, D>(p, dev, sms, st)
                                 : launch_pool<FORM, T, kPoolSame, D>(p, dev, sms, st);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

// What a rotating append is called with, plain or normed.
struct RopeCall {
    void* q_out;
    const void* q;
    int64_t q_stride;
    const void* k;
    int64_t k_stride;
    const void* v;
    int64_t v_stride;
    const int32_t* positions;
    const float* cos_sin;
    int32_t max_position, rot_dim, interleaved;
    void *k_pool, *v_pool;
    const int64_t* slot_mapping;
    int32_t num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
    pa_dtype in_dtype, pool_dtype;
    float k_scale, v_scale;
    int32_t* dev_status;
    void* stream;
    // normed form
    const float *q_weight, *k_weight;
    void* k_out;
    float eps;
};

template <typename FORM>
pa_status rope_call(const RopeCall& c) {
    if (c.num_tokens < 0 || c.num_q_heads < 0 || c.num_kv_heads <= 0 || c.num_blocks <= 0 || c.max_position <= 0 || c.rot_dim <= 0 ||
        (c.interleaved != 0 && c.interleaved != 1))
        return PA_ERR_INVALID_ARG;
    if (c.in_dtype != PA_F32 && c.in_dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    const bool quantised = c.pool_dtype == PA_FP8_E4M3 || c.pool_dtype == PA_FP4_E2M1;
    if (!quantised && c.pool_dtype != c.in_dtype) return PA_ERR_UNSUPPORTED;
    if ((c.head_dim != 64 && c.head_dim != 128) || (c.block_size != 16 && c.block_size != 32) ||
        (c.pool_dtype == PA_FP8_E4M3 && c.head_dim != 128))
        return PA_ERR_UNSUPPORTED;
    if (c.rot_dim > c.head_dim) return PA_ERR_INVALID_ARG;
    if (c.rot_dim % (c.pool_dtype == PA_FP4_E2M1 ? 32 : 16)) return PA_ERR_UNSUPPORTED;
    if (!std::isfinite(c.k_scale) || !std::isfinite(c.v_scale) || !(c.k_scale > 0.f) || !(c.v_scale > 0.f)) return PA_ERR_INVALID_ARG;
    const int64_t heads = (int64_t)c.num_q_heads + 2 * (int64_t)c.num_kv_heads;
    if (heads * c.num_tokens * (c.head_dim / 16) >= INT32_MAX / 2) return PA_ERR_UNSUPPORTED;
    const int64_t per16 = c.in_dtype == PA_F32 ? 4 : 8;  // elements in 16 bytes
    if ((c.num_q_heads > 0 && c.q_stride < (int64_t)c.num_q_heads * c.head_dim) || c.k_stride < (int64_t)c.num_kv_heads * c.head_dim ||
        c.v_stride < (int64_t)c.num_kv_heads * c.head_dim || (c.num_q_heads > 0 && c.q_stride % per16) || c.k_stride % per16 ||
        c.v_stride % per16)
        return PA_ERR_INVALID_ARG;
    if (c.num_tokens == 0) return PA_OK;
    if ((c.num_q_heads > 0 && (!c.q || !c.q_out)) || !c.k || !c.v || !c.positions || !c.cos_sin || !c.k_pool || !c.v_pool || !c.slot_mapping)
        return PA_ERR_INVALID_ARG;
    if ((c.num_q_heads > 0 && (!aligned16(c.q) || !aligned16(c.q_out))) || !aligned16(c.k) || !aligned16(c.v) || !aligned16(c.cos_sin) ||
        !aligned16(c.k_pool) || !aligned16(c.v_pool) || (reinterpret_cast<uintptr_t>(c.slot_mapping) & 7u) ||
        (reinterpret_cast<uintptr_t>(c.positions) & 3u) || (reinterpret_cast<uintptr_t>(c.dev_status) & 3u))
        return PA_ERR_INVALID_ARG;
    // queries in place must be laid out as c.q_out is
    if (c.num_q_heads > 0 && c.q == c.q_out && c.q_stride != (int64_t)c.num_q_heads * c.head_dim) return PA_ERR_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return PA_ERR_CUDA;
    RopeParams p;
    p.q_out = c.q_out, p.q = c.q, p.k = c.k, p.v = c.v;
    p.q_stride = c.q_stride, p.k_stride = c.k_stride, p.v_stride = c.v_stride;
    p.positions = c.positions;
    p.cos_sin = c.cos_sin;
    p.slots = c.slot_mapping;
    p.k_pool = static_cast<uint8_t*>(c.k_pool), p.v_pool = static_cast<uint8_t*>(c.v_pool);
    p.pool_slots = (int64_t)c.num_blocks * c.block_size;
    p.k_scale = divisor(c.k_scale), p.v_scale = divisor(c.v_scale);
    p.status = c.dev_status;
    p.num_tokens = c.num_tokens, p.num_q_heads = c.num_q_heads, p.num_kv_heads = c.num_kv_heads;
    p.bs_shift = c.block_size == 16 ? 4 : 5, p.max_position = c.max_position, p.rot_dim = c.rot_dim, p.interleaved = c.interleaved;
    p.heads = fast_div((uint32_t)heads);
    p.q_weight = c.q_weight, p.k_weight = c.k_weight, p.k_out = c.k_out, p.eps = c.eps;
    cudaStream_t st = static_cast<cudaStream_t>(c.stream);
    bool ok;
    if (c.in_dtype == PA_BF16)
        ok = c.head_dim == 128 ? launch_rope<FORM, __nv_bfloat16, 128>(p, c.pool_dtype, dev, sms, st)
                             : launch_rope<FORM, __nv_bfloat16, 64>(p, c.pool_dtype, dev, sms, st);
    else
        ok = c.head_dim == 128 ? launch_rope<FORM, float, 128>(p, c.pool_dtype, dev, sms, st)
                             : launch_rope<FORM, float, 64>(p, c.pool_dtype, dev, sms, st);
    if (!ok) return PA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa
