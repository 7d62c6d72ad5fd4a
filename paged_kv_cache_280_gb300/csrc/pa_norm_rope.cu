// Normed rotating append: every query and key head scaled to a unit mean of squares and by its weights, then turned and
// appended as the rotating append does.
//
// x of a head, r = 1 / sqrt(mean(x^2) + eps), w its weights; of a turned pair (a, b), c and s as in pa_rope.cuh:
//     a' = (a r) (wa c) - (b r) (wb s),   b' = (b r) (wb c) + (a r) (wa s),
// past rot_dim x' = (x r) w.  The four products of a pair's weights with c and s are the same for all query heads of a
// token and for all its key heads, so a thread keeps them: a warp takes rows (one head of one token) that lie one behind
// the other, first of queries, then of keys and values, and works its factors out where the token changes.
#include "pa_rope.cuh"

namespace pa {
namespace {

// Measured: 8191 tokens of 64 + 16 heads of 128, bf16 into FP8 pools, keys also stored dense (340 MB): 58.6 us, 5.8 TB/s (0.85
// of the measured copy rate; DRAM moves 296 MB, the rest is written back later).  With the weights and cos / sin applied one after the other and read for
// every row, as the plain append reads them, 75: the rows' shared-memory and issue slots bound it then, 302 instructions
// a warp's turn against 206; now it is memory latency.  Keys and values in the queries' loop: 59.6, but registers spill
// into the 4-bit pools.  CTAs per SM: 5 (96 registers, none spilled); 4: 62, 6: 66.  One wave of CTAs: 62, 2: 60, 4: 61.
// Three turns ahead: 68; a warp's rows not in one run but in many of 8 turns: 62, of 4: 66.
constexpr int kNormThreads = 128, kNormCtas = 5, kNormWarps = kNormThreads / 32, kNormWaves = 2;

__device__ __forceinline__ void prefetch_l1(const void* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void load4f(const float* p, float* x) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}

// A warp's share of the query rows, or (KV) of the key and value rows: R rows a turn, from row0 to row_end.
template <typename T, int POOL, int D, bool KV>
__device__ __forceinline__ void norm_rows(const RopeParams& p, uint32_t mine, const FastDiv heads, uint32_t row0, uint32_t row_end) {
    constexpr int U = D / 16, R = 32 / U;  // units of a row; rows of a warp's turn
    constexpr int kParts = (int)sizeof(T) / 2;
    constexpr uint32_t kPart = kNormThreads * 16, kTurn = 2 * kParts * kPart;
    const int H = (int)heads.d, half = p.rot_dim / 2;
    const int u = (int)(threadIdx.x & (U - 1));
    const bool rot_unit = 16 * u < p.rot_dim;
    const int e0 = rot_unit ? 8 * u : 8 * u + half;
    const int e1 = rot_unit ? 8 * u + half : 8 * u + half + (D - p.rot_dim) / 2;

    // A row's token and head, and where it is read.
    uint32_t row = row0 + (threadIdx.x & 31) / U, tok = heads.div(row), far_tok = tok;
    int h = (int)(row - tok * heads.d), far_h = h;
    const T* src = nullptr;
    T* dst = nullptr;
    auto settle_far = [&] {
        while (far_h >= H) far_h -= H, ++far_tok;
        if (KV)
            src = far_h < p.num_kv_heads ? static_cast<const T*>(p.k) + far_tok * p.k_stride + far_h * D
                                         : static_cast<const T*>(p.v) + far_tok * p.v_stride + (far_h - p.num_kv_heads) * D;
        else
            src = static_cast<const T*>(p.q) + far_tok * p.q_stride + far_h * D;
    };
    settle_far();
    auto fetch = [&](int turn, uint32_t far_row) {
        if (far_row < row_end) {
            const uint32_t to = mine + turn * kTurn;
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                copy_ahead16<kParts == 2>(to + i * kPart, src + e0 + 4 * i);
                copy_ahead16<kParts == 2>(to + (kParts + i) * kPart, src + e1 + 4 * i);
            }
        }
        copies_commit();
        const bool was_key = KV && far_h < p.num_kv_heads;
        far_h += R, src += R * D;
        if (far_h >= H || (was_key && far_h >= p.num_kv_heads)) settle_far();
    };
#pragma unroll
    for (int i = 0; i < kRopeAhead; ++i) fetch(i, row + i * R);

    // Of tok: its slot, whether it is appended, and the factors of its heads.
    int64_t slot = -1;
    bool ok = false;
    float ca[8], sb[8], cb[8], sa[8];  // wa c, wb s, wb c, wa s; past rot_dim wa and wb in ca and cb
    auto settle = [&] {
        while (h >= H) h -= H, ++tok;
        ok = row < row_end;
        if (!ok) return;
        if (!KV) dst = static_cast<T*>(p.q_out) + ((int64_t)tok * H + h) * D;
        slot = p.slots[tok];
        const int pos = p.positions[tok];  // (of a padding token: not looked at)
        if (tok + 1 < (uint32_t)p.num_tokens) prefetch_l1(p.slots + tok + 1), prefetch_l1(p.positions + tok + 1);
        ok = slot >= 0;
        if (!ok) return;
        const bool bad_slot = slot >= p.pool_slots, bad_pos = pos < 0 || pos >= p.max_position;
        if (bad_slot || bad_pos) {
            ok = false;
            if (KV && h == 0 && u == 0)
                flag_status(p.status, (bad_slot ? PA_DEV_BAD_SLOT : 0) | (bad_pos ? PA_DEV_BAD_POSITION : 0));
            return;
        }
        const float* w = KV ? p.k_weight : p.q_weight;
#pragma unroll
        for (int i = 0; i < 8; ++i) ca[i] = w[e0 + i], cb[i] = w[e1 + i];
        if (!rot_unit) return;
        const float* cs = p.cos_sin + (int64_t)pos * p.rot_dim;
        float c[8], s[8];
        if (p.interleaved) {  // four pairs of each run; the factors of the run at e0 in ca and sb, of that at e1 in cb and sa
#pragma unroll
            for (int i = 0; i < 2; ++i) load4f(cs + (i ? e1 : e0) / 2, c + 4 * i), load4f(cs + half + (i ? e1 : e0) / 2, s + 4 * i);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float wx = ca[2 * i], wy = ca[2 * i + 1], vx = cb[2 * i], vy = cb[2 * i + 1];
                ca[2 * i] = wx * c[i], ca[2 * i + 1] = wy * c[i], sb[2 * i] = wy * s[i], sb[2 * i + 1] = wx * s[i];
                cb[2 * i] = vx * c[4 + i], cb[2 * i + 1] = vy * c[4 + i], sa[2 * i] = vy * s[4 + i], sa[2 * i + 1] = vx * s[4 + i];
            }
        } else {
            load8(cs + e0, c);
            load8(cs + half + e0, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wa = ca[i], wb = cb[i];
                ca[i] = wa * c[i], sb[i] = wb * s[i], cb[i] = wb * c[i], sa[i] = wa * s[i];
            }
        }
    };
    settle();
    int turn = 0;
    // every thread of a warp takes the same number of turns: squares and 4-bit groups meet in shuffles
    for (uint32_t base = row0; base < row_end; base += R) {
        copies_wait<kRopeAhead - 1>();
        float a[8], b[8];
        take8<T>(mine + turn * kTurn, kPart, a);
        take8<T>(mine + turn * kTurn + kParts * kPart, kPart, b);
        fetch(turn, row + kRopeAhead * R);
        if (++turn == kRopeAhead) turn = 0;
        const bool is_v = KV && h >= p.num_kv_heads;
        // a row's units are U neighbouring lanes of one warp: the sum of its squares meets in shuffles
        float2 sq2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 x = make_float2(a[j], a[j + 1]), y = make_float2(b[j], b[j + 1]);
            sq2 = fma_f32x2(y, y, fma_f32x2(x, x, sq2));
        }
        float sq = sq2.x + sq2.y;
#pragma unroll
        for (int o = 1; o < U; o *= 2) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (!is_v) {
            const float r = __frsqrt_rn(sq * (1.f / D) + p.eps);
            const float2 rr = make_float2(r, r);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 x = mul_f32x2(make_float2(a[j], a[j + 1]), rr), y = mul_f32x2(make_float2(b[j], b[j + 1]), rr);
                const float2 fa = make_float2(ca[j], ca[j + 1]), fb = make_float2(cb[j], cb[j + 1]);
                float2 na = mul_f32x2(x, fa), nb = mul_f32x2(y, fb);
                if (rot_unit) {
                    const float2 ga = make_float2(sa[j], sa[j + 1]), gb = make_float2(sb[j], sb[j + 1]);
                    if (p.interleaved) {  // a pair's two side by side
                        na = fma_f32x2(make_float2(-x.y, x.x), gb, na);
                        nb = fma_f32x2(make_float2(-y.y, y.x), ga, nb);
                    } else {
                        na = fma_f32x2(make_float2(-y.x, -y.y), gb, na);
                        nb = fma_f32x2(x, ga, nb);
                    }
                }
                a[j] = na.x, a[j + 1] = na.y, b[j] = nb.x, b[j + 1] = nb.y;
            }
        }
        if (!KV) {
            if (ok) {
                store8(dst + e0, a);
                store8(dst + e1, b);
            }
            dst += R * D;
        } else {
            if (ok && !is_v && p.k_out) {
                T* to = static_cast<T*>(p.k_out) + ((int64_t)tok * p.num_kv_heads + h) * D;
                store8(to + e0, a);
                store8(to + e1, b);
            }
            append_unit<T, POOL, D>(p, ok, is_v, h - (is_v ? p.num_kv_heads : 0), slot, u, e0, e1, a, b);
        }
        row += R, h += R;
        if (h >= H) settle();
        if (row >= row_end) ok = false;
    }
}

template <typename T, int POOL, int D>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_rope_kernel(const RopeParams p) {
    pdl_wait_prerequisites();  // as in rope_and_cache_kernel
    pdl_launch_dependents();
    constexpr uint32_t R = 512 / D, kTurn = (uint32_t)sizeof(T) * kNormThreads * 16;
    __shared__ __align__(16) uint8_t ahead[kRopeAhead * kTurn];
    const uint32_t mine = smem_u32(ahead) + threadIdx.x * 16;
    const uint32_t warps = gridDim.x * kNormWarps, w = blockIdx.x * kNormWarps + threadIdx.x / 32;
    auto share = [&](uint32_t rows, uint32_t at, uint32_t& begin, uint32_t& end) {  // of warp number `at`
        const uint32_t turns = ((rows + R - 1) / R + warps - 1) / warps;
        begin = min(at * turns * R, rows), end = min(begin + turns * R, rows);
    };
    uint32_t begin, end;
    if (p.num_q_heads > 0) {
        share((uint32_t)p.num_tokens * (uint32_t)p.num_q_heads, w, begin, end);
        norm_rows<T, POOL, D, false>(p, mine, p.q_heads, begin, end);
    }
    // in the other order: of a small call's warps the first take queries, the last keys and values
    share((uint32_t)p.num_tokens * 2u * (uint32_t)p.num_kv_heads, warps - 1 - w, begin, end);
    norm_rows<T, POOL, D, true>(p, mine, p.kv_heads, begin, end);
}

struct NormRope {
    template <typename T, int POOL, int D>
    static auto kernel() { return &norm_rope_kernel<T, POOL, D>; }
    static constexpr int kThreads = kNormThreads;
    static unsigned grid(RopeParams& p, int64_t units, int resident) {
        if (p.num_q_heads > 0) p.q_heads = fast_div((uint32_t)p.num_q_heads);
        p.kv_heads = fast_div(2u * (uint32_t)p.num_kv_heads);
        const int64_t want = (units + kNormThreads - 1) / kNormThreads + 1;  // queries and the rest each end a warp's turn
        const int64_t most = kNormWaves * (int64_t)resident;
        return (unsigned)(want < most ? want : most);
    }
};

}  // namespace
}  // namespace pa

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
    return pa::rope_call<pa::NormRope>({q_out, q, q_stride, k, k_stride, v, v_stride, positions, cos_sin, max_position, rot_dim,
                                interleaved, k_pool, v_pool, slot_mapping, num_tokens, num_q_heads, num_kv_heads,
                                head_dim, block_size, num_blocks, in_dtype, pool_dtype, k_scale, v_scale, dev_status,
                                stream, q_weight, k_weight, k_out, eps});
}
