// Decode over 4-bit pools with bf16 queries and outputs, on the tensor cores for every group size.
//
// The arithmetic and its bound are in pa_decode_fp4.cuh: a warp spends about as many issue slots on a
// tile as HBM takes to deliver it, so this kernel is organised to have as many warps computing as fit
// and to spend nothing else.  Every warp is a worker of its own: it owns one range of the plan
// (pa_plan.h; what the other decode kernels call a CTA's range), copies its tiles into a private ring
// of kStages stages of 32 tokens (cp.async.bulk: a tile of this format is one contiguous record), and
// computes on them.  There is no producer warp, no hand-over between warps and no barrier after the
// prologue; a stage is refilled by the warp that has just read it.  Partials of split segments are
// merged by a second kernel, launched as the programmatic dependent of this one.
#include "pa_decode.cuh"
#include "pa_decode_fp4.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;    // workers per CTA
constexpr int kStages = 2;   // ring stages per worker
constexpr int kStageTok = 32;
constexpr int kMinCtasPerSm = 4;

template <int D, int BS>
struct Fp4Layout {
    static constexpr int TPS = kStageTok / BS;  // tiles per stage
    static constexpr int kTile = BS * fp4_row_bytes(D);
    static constexpr int kStageBytes = 2 * TPS * kTile;  // K of its tiles, then their V
    static constexpr int kDescOff = kWarps * kStages * kStageBytes;   // int4 per stage
    static constexpr int kBarOff = kDescOff + kWarps * kStages * 16;  // full barrier per stage
    static constexpr int kWsumOff = kBarOff + kWarps * kStages * 8;
    static constexpr int kPrefixOff = (kWsumOff + 2 * kWarps * 4 + 15) / 16 * 16;
    static_assert(kStageBytes % 16 == 0, "bulk-copy alignment");
    static constexpr int bytes(int num_seqs, bool fixed) {
        return kPrefixOff + (num_seqs + 1) * 4 * (fixed ? 2 : 1) + num_seqs * 4 + 16;
    }
};

// The plan of this launch over the scanned batch: fp4_ranges() of p.num_ctas ranges take work.
template <int BS>
__device__ __forceinline__ Plan fp4_plan(const DecodeParams& p, const int32_t* pref, const int32_t* upref) {
    const int64_t tiles = (int64_t)p.num_kv_heads * pref[p.num_seqs];
    return plan_from_prefix(pref, upref, p.num_seqs, p.num_kv_heads, p.partition_tiles, p.seg_units,
                            fp4_ranges(tiles, p.num_ctas, p.partition_tiles, BS), p.wave_ctas, p.wave_skew);
}

// As plan_matches, for a plan built for a 4-bit pool (its magic word differs, since its ranges do).
__device__ __forceinline__ bool fp4_plan_matches(const DecodeParams& p, int bs) {
    const int32_t* pl = p.plan;
    if (pl == nullptr) return false;
    return __ldg(pl + kPlanWMagic) == kPlanMagicFp4 && __ldg(pl + kPlanWNumSeqs) == p.num_seqs &&
           __ldg(pl + kPlanWGrid) == p.num_ctas && __ldg(pl + kPlanWKvHeads) == p.num_kv_heads &&
           __ldg(pl + kPlanWPartitionTiles) == p.partition_tiles && __ldg(pl + kPlanWSegUnits) == p.seg_units &&
           __ldg(pl + kPlanWBlockSize) == bs && __ldg(pl + kPlanWMaxLen) == p.max_len &&
           __ldg(pl + kPlanWMergeInKernel) == p.merge_in_kernel &&
           __ldg(pl + kPlanWMaxBlocks) == p.max_blocks_per_seq && __ldg(pl + kPlanWWaveCtas) == p.wave_ctas &&
           __ldg(pl + kPlanWWaveSkew) == p.wave_skew;
}

// How the merge enumerates its items (see merge_fp4_kernel).
__host__ __device__ inline bool fp4_merge_wide(int num_seqs, int num_kv_heads, int ranges) {
    return (int64_t)num_seqs * num_kv_heads <= ranges;
}

enum StageFlag { kFirst = 64, kLast = 128, kWhole = 256, kSlot1 = 512 };  // beside the valid tokens (1 .. 32)

template <int D, int BS>
__global__ void __launch_bounds__(32 * kWarps, kMinCtasPerSm) decode_fp4_kernel(const DecodeParams p) {
    using L = Fp4Layout<D, BS>;
    constexpr int TPS = L::TPS;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs, Hkv = p.num_kv_heads, Hq = p.num_q_heads, G = p.group;
    const int c = blockIdx.x * kWarps + warp;  // the worker
    const bool fixed = p.partition_tiles > 0;
    int32_t* pref = reinterpret_cast<int32_t*>(smem + L::kPrefixOff);
    int32_t* upref = pref + (B + 1);
    int32_t* lens_s = upref + (fixed ? B + 1 : 0);
    int32_t* wsum = reinterpret_cast<int32_t*>(smem + L::kWsumOff);
    const uint32_t ring = smem_u32(smem) + warp * kStages * L::kStageBytes;
    const uint32_t bar = smem_u32(smem) + L::kBarOff + warp * kStages * 8;
    int4* desc = reinterpret_cast<int4*>(smem + L::kDescOff) + warp * kStages;

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
        fence_barrier_init();
    }
    bool planned = false;
    int32_t rec = 0, first_chunk = 0;
    int32_t pw[kPlanPass];
    if (p.plan != nullptr) {
        if (c < p.num_ctas) {
            const int32_t* r = p.plan + plan_rec_off(B, c);
            if (lane < kRecFirst) rec = __ldg(r + lane);
            first_chunk = __ldg(r + kRecFirst + lane);
        }
        plan_words_load<32 * kWarps>(p, 0, pw);
        planned = fp4_plan_matches(p, BS);
    }
    if (planned)
        load_plan_arrays<32 * kWarps>(p, pw, pref, upref, lens_s);
    else
        scan_lengths<BS, 32 * kWarps>(p, blockIdx.x == 0, pref, upref, lens_s, wsum);
    __syncthreads();
    const Plan P = fp4_plan<BS>(p, pref, upref);
    pdl_launch_dependents();
    const bool works = P.T > 0 && c < P.C;
    int64_t tb = 0, split = -1;
    int seqh = 0;
    if (!planned && works && lane < 2) tb = P.cta_start(c + lane, &split, &seqh);
    const int32_t t0 = planned ? __shfl_sync(0xffffffffu, rec, kRecT0) : (int32_t)__shfl_sync(0xffffffffu, tb, 0);
    const int32_t t1 = planned ? __shfl_sync(0xffffffffu, rec, kRecT1) : (int32_t)__shfl_sync(0xffffffffu, tb, 1);
    const int seq0 = planned ? __shfl_sync(0xffffffffu, rec, kRecSeq0) : __shfl_sync(0xffffffffu, seqh, 0);

    // The walk of the copies, kStages stages ahead of the computation.
    const uint64_t policy = policy_evict_first();
    PieceIter<false> it;
    it.init(P, t0, works ? t1 : t0, -1, seq0, seq0);
    int b = 0, h = 0, j0 = 0, j1 = 0, j = 0, len = 0, nb = 0;
    int32_t blk = 0;  // table entries of 32 tiles of the piece, the first at jc
    int jc = 0;
    auto next_piece = [&]() -> bool {
        if (!it.next(P, b, h, j0, j1)) return false;
        j = j0;
        len = lens_s[b];
        nb = P.nblocks(b);
        return true;
    };
    auto load_chunk = [&]() {
        jc = j;
        blk = j + lane < j1 ? __ldg(p.block_tables + (size_t)b * p.max_blocks_per_seq + j + lane) : 0;
    };
    bool have = next_piece();
    if (have) {
        if (planned) {
            jc = j;
            blk = first_chunk;
        } else {
            load_chunk();
        }
    }
    pdl_wait_prerequisites();  // pools, q and out from here on
    for (int bb = c; bb < B; bb += p.num_ctas) {
        if (pref[bb + 1] == pref[bb]) {  // an empty sequence
            uint32_t* o = static_cast<uint32_t*>(p.out) + (size_t)bb * Hq * (D / 2);
            for (int e = lane; e < Hq * (D / 2); e += 32) o[e] = 0;
        }
    }
    // Copy the next stage of the walk into ring slot s (whose previous contents this warp has read).
    auto issue = [&](int s) {
        const int nt = min(TPS, j1 - j);
        const int t = lane % TPS;
        int32_t bid = __shfl_sync(0xffffffffu, blk, (j - jc + t) & 31);
        if (t < nt && (bid < 0 || bid >= p.num_blocks)) {
            if (lane < TPS) flag_status(p.status, PA_DEV_BAD_BLOCK_ID);
            bid = 0;
        }
        if (lane == 0) {
            const int flags = (j == j0 ? kFirst : 0) | (j + nt == j1 ? kLast : 0) | (j0 == 0 && j1 == nb ? kWhole : 0) |
                              (j0 == 0 ? kSlot1 : 0);
            desc[s] = make_int4(min(nt * BS, len - j * BS) | flags, b, h, 0);
            mbar_arrive_expect_tx(bar + 8 * s, (uint32_t)(nt * 2 * L::kTile));
        }
        __syncwarp();
        if (lane < 2 * TPS && t < nt)
            bulk_load_hint(ring + s * L::kStageBytes + lane * L::kTile,
                           (lane < TPS ? p.k_pool : p.v_pool) + ((int64_t)bid * Hkv + h) * L::kTile, L::kTile, bar + 8 * s,
                           policy);
        j += nt;
        if (j == j1) {
            have = next_piece();
            if (have) load_chunk();
        } else if (j - jc == 32) {
            load_chunk();
        }
    };
    uint32_t issued = 0, used = 0;
#pragma unroll 1
    for (int s = 0; s < kStages && have; ++s, ++issued) issue(s);

    Fp4State<D, BS> st;
    bool ok = true;
    int s = 0;
    uint32_t parity = 0;
    while (used < issued) {
        const int4 d = desc[s];
        if (d.x & kFirst) {
            st.load_q(static_cast<const __nv_bfloat16*>(p.q) + ((size_t)d.y * Hq + (size_t)d.z * G) * D, G, lane,
                      p.scale_log2);
            st.reset();
        }
        ok = __all_sync(0xffffffffu, mbar_wait(bar + 8 * s, parity, p.wait_limit_ns));
        if (!ok) break;
        const uint32_t kb = ring + s * L::kStageBytes;
        st.stage(kb, kb + TPS * L::kTile, d.x & 63, lane);
        __syncwarp();
        ++used;
        if (have) {
            issue(s);
            ++issued;
        }
        if (++s == kStages) s = 0, parity ^= 1;
        if (d.x & kLast) {
            if (d.x & kWhole)
                st.store_out(static_cast<__nv_bfloat16*>(p.out) + ((size_t)d.y * Hq + (size_t)d.z * G) * D, G, lane, p.out_scale);
            else  // slot 1: a split segment's first piece; slot 0: one that continues it
                st.store_partial(p.partials + (size_t)(2 * c + (d.x & kSlot1 ? 1 : 0)) * partial_slot_floats(G, D), G, lane);
        }
    }
    if (!ok) {
        // a wait gave up: the output is not valid, but no copy may land after the CTA has gone
        if (lane == 0) flag_status(p.status, PA_DEV_WAIT_TIMEOUT);
        for (; used < issued; ++used) {
            mbar_wait(bar + 8 * s, parity);
            if (++s == kStages) s = 0, parity ^= 1;
        }
    }
}

// The merge of split segments: M = max m_p, out = sum 2^(m_p - M) o_p / sum 2^(m_p - M) l_p over a
// segment's pieces.  An item is one query head of one segment.  With no more segments than ranges
// (long contexts: many pieces each) the items are enumerated by segment and the four warps of a CTA
// share an item's pieces; with more (most segments whole, a split one in two or three pieces) they
// are enumerated by range boundary, the first boundary inside a segment naming it, a warp to an item.
// The loads of four pieces are in flight together.  Pieces are folded in a fixed order: a call's
// result does not depend on timing.
template <int D, int BS>
__global__ void __launch_bounds__(kMergeThreads) merge_fp4_kernel(const DecodeParams p) {
    extern __shared__ __align__(16) int32_t msm[];
    constexpr int E = D / 32;  // output elements per lane
    constexpr int kW = kMergeThreads / 32;
    __shared__ float part[kW][D + 2];
    const int B = p.num_seqs, Hkv = p.num_kv_heads, G = p.group;
    const bool fixed = p.partition_tiles > 0;
    int32_t* pref = msm;
    int32_t* upref = pref + (B + 1);
    int32_t* lens_s = upref + (fixed ? B + 1 : 0);
    int32_t* wsum = lens_s + B;
    int32_t pw[kPlanPass];
    if (p.plan != nullptr) plan_words_load<kMergeThreads>(p, 0, pw);  // in bounds: the host checked its size
    if (fp4_plan_matches(p, BS))
        load_plan_arrays<kMergeThreads>(p, pw, pref, upref, lens_s);
    else
        scan_lengths<BS, kMergeThreads>(p, false, pref, upref, lens_s, wsum);
    __syncthreads();
    const Plan P = fp4_plan<BS>(p, pref, upref);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t slot_floats = partial_slot_floats(G, D);
    const bool wide = fp4_merge_wide(B, Hkv, p.num_ctas);
    const int step = wide ? kW : 1, first = wide ? warp : 0;  // this warp's pieces of an item
    const int64_t items = wide ? (int64_t)B * Hkv * G : (int64_t)(P.C - 1) * G;
    const int64_t stride = (int64_t)gridDim.x * (wide ? 1 : kW);
    int64_t item = wide ? blockIdx.x : (int64_t)blockIdx.x * kW + warp;
    // the item's sequence, KV head, first range and pieces; false if its segment is not split (or named elsewhere)
    auto named = [&](int64_t i, int& b, int& h, int& ca, int& np) -> bool {
        if (wide) {
            const int seg = (int)(i / G);
            b = seg / Hkv;
            h = seg - b * Hkv;
            const int nb = P.nblocks(b);
            if (nb == 0) return false;
            const int64_t s0 = P.seg_start(b, h);
            ca = P.cta_of_seg(s0, b, h);
            np = P.cta_of_seg(s0 + nb - 1, b, h) - ca + 1;
            return np > 1;
        }
        int64_t split;
        int seq;
        const int c = 1 + (int)(i / G);
        const int64_t t = P.cta_start(c, &split, &seq);
        if (t >= P.T) return false;
        b = P.find_seq(P.pref, t);
        const int nb = P.nblocks(b);
        const int64_t local = t - (int64_t)Hkv * P.pref[b];
        h = (int)(local / nb);
        if (local == (int64_t)h * nb) return false;  // the boundary falls between segments
        const int64_t s0 = (int64_t)Hkv * P.pref[b] + (int64_t)h * nb;
        ca = P.cta_of_seg(s0, b, h);
        if (ca != c - 1) return false;  // an earlier boundary of this segment names it
        np = P.cta_of_seg(s0 + nb - 1, b, h) - ca + 1;
        return true;
    };
    int b = 0, h = 0, ca = 0, np = 0;
    bool have = P.T > 0 && item < items && named(item, b, h, ca, np);  // found while the decode runs
    pdl_wait_prerequisites();  // the decode grid has finished; its partials are in memory
    while (P.T > 0 && item < items) {
        if (have) {
            const int hq = (int)(item % G);
            float m = -INFINITY, l = 0.f, a[E];
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = 0.f;
            for (int i0 = first; i0 < np; i0 += 4 * step) {
                float2 ml[4];
                float x[4][E];
                float mc = m;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int q = i0 + i * step;
                    if (q < np) {
                        const float* sp = piece_slot(p.partials, slot_floats, ca + q, ca);
                        ml[i] = __ldcg(reinterpret_cast<const float2*>(sp + G * D) + hq);
                        if constexpr (E == 4) {
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(sp + hq * D) + lane);
                            x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
                        } else {
                            const float2 v = __ldcg(reinterpret_cast<const float2*>(sp + hq * D) + lane);
                            x[i][0] = v.x, x[i][1] = v.y;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i * step < np) mc = fmaxf(mc, ml[i].x);
                const float resc = m == mc ? 1.f : ex2_approx(m - mc);
                l *= resc;
#pragma unroll
                for (int e = 0; e < E; ++e) a[e] *= resc;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i * step < np) {
                        const float w = ex2_approx(ml[i].x - mc);
                        l = fmaf(w, ml[i].y, l);
#pragma unroll
                        for (int e = 0; e < E; ++e) a[e] = fmaf(w, x[i][e], a[e]);
                    }
                m = mc;
            }
            if (wide) {
                // fold the warps' sums, in warp order
                __syncthreads();
                if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
#pragma unroll
                for (int e = 0; e < E; ++e) part[warp][E * lane + e] = a[e];
                __syncthreads();
                if (warp == 0) {
                    float mc = m;
                    for (int w = 1; w < kW && w < np; ++w) mc = fmaxf(mc, part[w][D]);
                    const float r0 = m == mc ? 1.f : ex2_approx(m - mc);
                    l *= r0;
#pragma unroll
                    for (int e = 0; e < E; ++e) a[e] *= r0;
                    for (int w = 1; w < kW && w < np; ++w) {
                        const float f = ex2_approx(part[w][D] - mc);
                        l = fmaf(f, part[w][D + 1], l);
#pragma unroll
                        for (int e = 0; e < E; ++e) a[e] = fmaf(f, part[w][E * lane + e], a[e]);
                    }
                }
            }
            if (!wide || warp == 0) {
                const float r = p.out_scale / l;
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) +
                                   ((size_t)b * p.num_q_heads + (size_t)h * G + hq) * D + E * lane;
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<uint32_t*>(o + e) = pack_bf16x2(a[e] * r, a[e + 1] * r);
            }
        }
        item += stride;
        have = item < items && named(item, b, h, ca, np);
    }
}

template <int D, int BS>
struct Fp4Variant {
    using L = Fp4Layout<D, BS>;
    static int smem(int num_seqs, bool fixed) { return L::bytes(num_seqs, fixed); }
    // grid: workers (ranges); kWarps to a CTA
    static void launch(const DecodeParams& p, const CUtensorMap&, const CUtensorMap&, int grid, int smem_bytes, int /*merge_grid*/,
                       int merge_smem, cudaStream_t stream) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((grid + kWarps - 1) / kWarps);
        cfg.blockDim = dim3(32 * kWarps);
        cfg.dynamicSmemBytes = smem_bytes;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, decode_fp4_kernel<D, BS>, p) != cudaSuccess) return;
        cudaLaunchConfig_t mcfg = cfg;
        const int sms = p.wave_ctas / kWarps;
        const int64_t items = fp4_merge_wide(p.num_seqs, p.num_kv_heads, grid)
                                  ? (int64_t)p.num_seqs * p.num_kv_heads * p.group
                                  : ((int64_t)(grid - 1) * p.group + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
        const int64_t most = (int64_t)sms * 8;
        mcfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < most ? items : most));
        mcfg.blockDim = dim3(kMergeThreads);
        mcfg.dynamicSmemBytes = merge_smem;
        cudaLaunchKernelEx(&mcfg, merge_fp4_kernel<D, BS>, p);
    }
    static DecodeVariant get() {
        const DecodeBuild b{reinterpret_cast<const void*>(&decode_fp4_kernel<D, BS>), kStages, 32 * kWarps, &smem};
        DecodeVariant v{b, b, reinterpret_cast<const void*>(&merge_fp4_kernel<D, BS>), false, &launch};
        v.ranges_per_cta = kWarps;
        return v;
    }
};

}  // namespace

bool decode_variant_fp4(int head_dim, int block_size, int group, DecodeVariant* out) {
    if (head_dim == 128 && block_size == 16) *out = Fp4Variant<128, 16>::get();
    else if (head_dim == 128 && block_size == 32) *out = Fp4Variant<128, 32>::get();
    else if (head_dim == 64 && block_size == 16) *out = Fp4Variant<64, 16>::get();
    else if (head_dim == 64 && block_size == 32) *out = Fp4Variant<64, 32>::get();
    else return false;
    return true;
}

}  // namespace pa
