// Decode over 4-bit pools with bf16 queries and outputs, on the tensor cores for every group size.
//
// The arithmetic and its bound are in pa_decode_fp4.cuh: a warp spends about as many issue slots on a
// tile as HBM takes to deliver it, so this kernel is organised to have as many warps computing as fit
// and to spend nothing else.  One CTA per SM owns one range of the plan (pa_plan.h); its kWarps warps cut
// the range into as many parts of equal cost, and each warp is on its own from there: it copies its
// tiles into a private ring of kStages stages of 32 tokens (cp.async.bulk: a tile of this format is one
// contiguous record) and computes on them.  There is no producer warp, no hand-over and no barrier
// while the range streams; a stage is refilled by the warp that has just read it.
//
// Pieces (the part of one (sequence, KV head) segment in one warp's part) that are whole segments are
// written straight to out.  The others meet in shared memory when all warps are done: runs of them
// that make up a segment are merged and written to out, a run that goes on in the next CTA or came from
// the one before becomes the CTA's partial in the workspace, and a second kernel, launched as the
// programmatic dependent of this one, merges those.
#include "pa_decode.cuh"
#include "pa_decode_fp4.cuh"

namespace pa {
namespace {

constexpr int kStages = 2;   // ring stages per warp
constexpr int kStageTok = 32;
constexpr size_t partial_slot_bytes_max(int d) { return (size_t)(kMaxGroup * (d + kSlotExtraFloatsPerHead) + 3) / 4 * 16; }

// What a warp has left of a segment at the end of its part: slot 0 a piece that continues a segment, slot
// 1 a segment's first piece, if the segment goes on.
struct Fp4Left {
    int32_t b, h;
    int32_t kind;  // 0 none; else bit 0: the segment starts in this piece, bit 1: it ends in it
    int32_t pad;
};

// kWarps: 16, one CTA per SM (512 threads of 128 registers), or 8 where a batch's prefix arrays leave no
// room for 16 rings.
template <int D, int BS, int kWarps>
struct Fp4Layout {
    static constexpr int TPS = kStageTok / BS;  // tiles per stage
    static constexpr int kTile = BS * fp4_row_bytes(D);
    static constexpr int kStageBytes = 2 * TPS * kTile;  // K of its tiles, then their V
    static constexpr int kRing = kStages * kStageBytes;  // per warp; slot 1's state goes here once the ring is idle
    static constexpr int kDescOff = kWarps * kRing;                  // int2 per stage
    static constexpr int kBarOff = kDescOff + kWarps * kStages * 8;  // full barrier per stage
    static constexpr int kLeftOff = (kBarOff + kWarps * kStages * 8 + 15) / 16 * 16;  // Fp4Left [kWarps][2]
    static constexpr int kWsumOff = kLeftOff + kWarps * 2 * 16;
    static constexpr int kSlot0Off = (kWsumOff + 2 * kWarps * 4 + 15) / 16 * 16;  // [kWarps][partial_slot_floats]
    static_assert(kTile % 16 == 0, "bulk-copy alignment");
    static_assert(kRing >= (int)partial_slot_bytes_max(D), "slot 1's state fits in the ring");
    static __host__ __device__ int prefix_off(int G) { return kSlot0Off + kWarps * (int)partial_slot_floats(G, D) * 4; }
    static int bytes(int G, int num_seqs, bool fixed) {
        return prefix_off(G) + (num_seqs + 1) * 4 * (fixed ? 2 : 1) + num_seqs * 4;
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

// A stage's descriptor: x = valid tokens (1 .. 32) | flags | KV head << 16, y = sequence.
enum StageFlag { kFirst = 64, kLast = 128, kStarts = 256, kEnds = 512 };

// Sum of a run of pieces for one query head: lane `lane` holds D / 32 elements.
template <int E>
struct Fp4Sum {
    float m = -INFINITY, l = 0.f, a[E];
    __device__ __forceinline__ Fp4Sum() {
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = 0.f;
    }
    __device__ __forceinline__ void add(float om, float ol, const float* oa) {
        const float mc = fmaxf(m, om);
        const float f = m == mc ? 1.f : ex2_approx(m - mc), w = om == mc ? 1.f : ex2_approx(om - mc);
        l = l * f + w * ol;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = a[e] * f + w * oa[e];
        m = mc;
    }
    __device__ __forceinline__ void store_out(__nv_bfloat16* row, int lane, float oscale) const {
        const float r = oscale / l;
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(row + E * lane + e) = pack_bf16x2(a[e] * r, a[e + 1] * r);
    }
};

template <int D, int BS, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) decode_fp4_kernel(const DecodeParams p) {
    using L = Fp4Layout<D, BS, kWarps>;
    constexpr int TPS = L::TPS, NT = 32 * kWarps;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = p.num_seqs, Hkv = p.num_kv_heads, Hq = p.num_q_heads, G = p.group, c = blockIdx.x;
    const bool fixed = p.partition_tiles > 0;
    const size_t slot_floats = partial_slot_floats(G, D);
    int32_t* pref = reinterpret_cast<int32_t*>(smem + L::prefix_off(G));
    int32_t* upref = pref + (B + 1);
    int32_t* lens_s = upref + (fixed ? B + 1 : 0);
    int32_t* wsum = reinterpret_cast<int32_t*>(smem + L::kWsumOff);
    float* slot0 = reinterpret_cast<float*>(smem + L::kSlot0Off);
    Fp4Left* left = reinterpret_cast<Fp4Left*>(smem + L::kLeftOff);
    const uint32_t ring = smem_u32(smem) + warp * L::kRing;
    const uint32_t bar = smem_u32(smem) + L::kBarOff + warp * kStages * 8;
    int2* desc = reinterpret_cast<int2*>(smem + L::kDescOff) + warp * kStages;

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
        fence_barrier_init();
        left[2 * warp].kind = left[2 * warp + 1].kind = 0;
    }
    int32_t pw[kPlanPass];
    if (p.plan != nullptr) plan_words_load<NT>(p, 0, pw);
    if (fp4_plan_matches(p, BS))
        load_plan_arrays<NT>(p, pw, pref, upref, lens_s);
    else
        scan_lengths<BS, NT>(p, c == 0, pref, upref, lens_s, wsum);
    __syncthreads();
    const Plan P = fp4_plan<BS>(p, pref, upref);
    pdl_launch_dependents();
    // this warp's part of the CTA's range, and a sequence at or before its start: two searches, lanes 0 and 1
    int64_t tb = 0, split = -1;
    int seqh = 0;
    if (P.T > 0 && c < P.C && lane < 2) {
        const int w = warp + lane;
        if (!fixed) {
            const int64_t u0 = P.start_unit(c), u1 = P.start_unit(c + 1), x = u0 + (u1 - u0) * w / kWarps;
            tb = c + 1 == P.C && w == kWarps ? P.T : P.first_tile_at_unit(x, &split, &seqh);
        } else {
            const int64_t r0 = P.cta_start(c, &split, &seqh);
            int dummy;
            const int64_t r1 = P.cta_start(c + 1, &split, &dummy);
            tb = r0 + (r1 - r0) * w / kWarps;
        }
    }
    const int32_t t0 = (int32_t)__shfl_sync(0xffffffffu, tb, 0), t1 = (int32_t)__shfl_sync(0xffffffffu, tb, 1);
    const int seq0 = __shfl_sync(0xffffffffu, seqh, 0);

    // The walk of the copies, kStages stages ahead of the computation.  Whatever stays the same within a
    // piece or a chunk of 32 table entries is worked out when they change: a stage then costs a few
    // instructions beside its copies.
    const uint64_t policy = policy_evict_first();
    PieceIter<false> it;
    it.init(P, t0, t1, -1, seq0, seq0);
    int b = 0, j = 0, j1 = 0, rem = 0, pflags = 0;  // sequence; next tile, end tile; tokens from tile j on; flags
    const uint8_t *kp = nullptr, *vp = nullptr;     // the pools at the piece's head
    int32_t blk = 0;                                // lane i: the block of tile i of the chunk
    int ci = 0;                                     // next tile within the chunk
    auto load_chunk = [&]() {
        ci = 0;
        blk = 0;
        if (j + lane < j1) {
            blk = __ldg(p.block_tables + (size_t)b * p.max_blocks_per_seq + j + lane);
            if ((uint32_t)blk >= (uint32_t)p.num_blocks) {
                flag_status(p.status, PA_DEV_BAD_BLOCK_ID);
                blk = 0;
            }
        }
    };
    auto next_piece = [&]() -> bool {
        int h, j0;
        if (!it.next(P, b, h, j0, j1)) return false;
        j = j0;
        rem = lens_s[b] - j0 * BS;
        pflags = kFirst | (j0 == 0 ? kStarts : 0) | (j1 == P.nblocks(b) ? kEnds : 0) | h << 16;
        kp = p.k_pool + (size_t)h * L::kTile;
        vp = p.v_pool + (size_t)h * L::kTile;
        load_chunk();
        return true;
    };
    bool have = next_piece();
    pdl_wait_prerequisites();  // pools, q and out from here on
    for (int bb = c * kWarps + warp; bb < B; bb += gridDim.x * kWarps) {
        if (pref[bb + 1] == pref[bb]) {  // an empty sequence
            uint32_t* o = static_cast<uint32_t*>(p.out) + (size_t)bb * Hq * (D / 2);
            for (int e = lane; e < Hq * (D / 2); e += 32) o[e] = 0;
        }
    }
    const uint32_t block_bytes = (uint32_t)Hkv * L::kTile;  // < 2^31 (checked on the host)
    // Copy the walk's next stage into ring slot s (whose previous contents this warp has read).
    auto issue = [&](int s) {
        const int nt = TPS == 1 ? 1 : min(TPS, j1 - j);
        const bool last = j + nt == j1;
        const uint64_t o0 = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, blk, ci) * block_bytes;
        const uint64_t o1 = TPS == 1 ? 0 : (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, blk, (ci + 1) & 31) * block_bytes;
        if (elect_one()) {
            desc[s] = make_int2(min(nt * BS, rem) | pflags | (last ? kLast : 0), b);
            const uint32_t full = bar + 8 * s, dst = ring + s * L::kStageBytes;
            mbar_arrive_expect_tx(full, (uint32_t)(nt * 2 * L::kTile));
            bulk_load_hint(dst, kp + o0, L::kTile, full, policy);
            bulk_load_hint(dst + TPS * L::kTile, vp + o0, L::kTile, full, policy);
            if (TPS > 1 && nt > 1) {
                bulk_load_hint(dst + L::kTile, kp + o1, L::kTile, full, policy);
                bulk_load_hint(dst + (TPS + 1) * L::kTile, vp + o1, L::kTile, full, policy);
            }
        }
        __syncwarp();
        pflags &= ~kFirst;
        j += nt;
        rem -= nt * BS;
        ci += nt;
        if (last)
            have = next_piece();
        else if (ci == 32)
            load_chunk();
    };
    uint32_t issued = 0, used = 0;
#pragma unroll 1
    for (int s = 0; s < kStages && have; ++s, ++issued) issue(s);

    Fp4State<D, BS> st;
    bool ok = true;
    int s = 0;
    uint32_t parity = 0;
    while (used < issued) {
        const int2 d = desc[s];
        const int sh = d.x >> 16, valid = d.x & 63;
        if (d.x & kFirst) {
            st.load_q(static_cast<const __nv_bfloat16*>(p.q) + ((size_t)d.y * Hq + (size_t)sh * G) * D, G, lane, p.scale_log2);
            st.reset();
        }
        if (!__all_sync(0xffffffffu, mbar_test_wait(bar + 8 * s, parity))) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar + 8 * s, parity, p.wait_limit_ns));
            if (!ok) break;
        }
        const uint32_t kb = ring + s * L::kStageBytes, vb = kb + TPS * L::kTile;
        uint32_t pb[4];
        if (valid == kStageTok) {
            st.template weights<false>(kb, valid, lane, pb);
            st.template accumulate<false>(vb, valid, lane, pb);
        } else {
            st.template weights<true>(kb, valid, lane, pb);
            st.template accumulate<true>(vb, valid, lane, pb);
        }
        __syncwarp();
        ++used;
        if (have) {
            issue(s);
            ++issued;
        }
        if (++s == kStages) s = 0, parity ^= 1;
        if (d.x & kLast) {
            const int kind = (d.x & kStarts ? 1 : 0) | (d.x & kEnds ? 2 : 0);
            if (kind == 3) {
                st.store_out(static_cast<__nv_bfloat16*>(p.out) + ((size_t)d.y * Hq + (size_t)sh * G) * D, G, lane, p.out_scale);
            } else {
                // a segment's first piece that does not end it is the warp's last piece: the ring is idle
                const int slot = kind == 1 ? 1 : 0;
                st.store_partial(slot ? reinterpret_cast<float*>(smem + warp * L::kRing) : slot0 + warp * slot_floats, G, lane);
                if (lane == 0) left[2 * warp + slot] = Fp4Left{d.y, sh, kind | 4, 0};
            }
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
    __syncthreads();
    // Runs of pieces of one segment, in warp order: a run opens with a piece in slot 1, or with the CTA's first
    // piece, and goes on through the following warps' slot 0.  One warp per (run, head).
    constexpr int E = D / 32;
    int item = 0;
    for (int i = 0; i < 2 * kWarps; ++i) {  // slots in order: warp 0's slot 0, its slot 1, ...
        const Fp4Left f = left[i];
        if (f.kind == 0) continue;
        // the run goes on through the slots 0 of the warps up to wl; a warp without a part has none
        const int w0 = i >> 1;
        int wl = w0, ends = f.kind & 2;
        for (int w = w0 + 1; w < kWarps && !ends; ++w) {
            const int kind = left[2 * w].kind;
            if (kind == 0) continue;
            ends = kind & 2;
            wl = w;
        }
        for (int hq = 0; hq < G; ++hq, ++item) {
            if (item % kWarps != warp) continue;
            Fp4Sum<E> sum;
            for (int w = w0; w <= wl; ++w) {
                if (w > w0 && left[2 * w].kind == 0) continue;
                const float* src = w == w0 && (i & 1) ? reinterpret_cast<const float*>(smem + w0 * L::kRing)
                                                      : slot0 + w * slot_floats;
                const float2 ml = *reinterpret_cast<const float2*>(src + G * D + 2 * hq);
                float x[E];
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = src[hq * D + E * lane + e];
                sum.add(ml.x, ml.y, x);
            }
            if ((f.kind & 1) && ends) {
                sum.store_out(static_cast<__nv_bfloat16*>(p.out) + ((size_t)f.b * Hq + (size_t)f.h * G + hq) * D, lane,
                              p.out_scale);
            } else {  // slot 1: a split segment's first piece; slot 0: one that continues it
                float* dst = p.partials + (size_t)(2 * c + (f.kind & 1)) * slot_floats;
#pragma unroll
                for (int e = 0; e < E; ++e) dst[hq * D + E * lane + e] = sum.a[e];
                if (lane == 0) dst[G * D + 2 * hq] = sum.m, dst[G * D + 2 * hq + 1] = sum.l;
            }
        }
        if (wl > w0) i = 2 * wl;  // the slots 0 up to wl are taken
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

template <int D, int BS, int kWarps>
struct Fp4Variant {
    using L = Fp4Layout<D, BS, kWarps>;
    template <int G>
    static int smem(int num_seqs, bool fixed) { return L::bytes(G, num_seqs, fixed); }
    static void launch(const DecodeParams& p, const CUtensorMap&, const CUtensorMap&, int grid, int smem_bytes, int /*merge_grid*/,
                       int merge_smem, cudaStream_t stream) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(32 * kWarps);
        cfg.dynamicSmemBytes = smem_bytes;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, decode_fp4_kernel<D, BS, kWarps>, p) != cudaSuccess) return;
        cudaLaunchConfig_t mcfg = cfg;
        const int64_t items = fp4_merge_wide(p.num_seqs, p.num_kv_heads, grid)
                                  ? (int64_t)p.num_seqs * p.num_kv_heads * p.group
                                  : ((int64_t)(grid - 1) * p.group + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
        const int64_t most = (int64_t)p.wave_ctas * 8;  // (wave_ctas: the SM count)
        mcfg.gridDim = dim3((unsigned)(items < 1 ? 1 : items < most ? items : most));
        mcfg.blockDim = dim3(kMergeThreads);
        mcfg.dynamicSmemBytes = merge_smem;
        cudaLaunchKernelEx(&mcfg, merge_fp4_kernel<D, BS>, p);
    }
    static DecodeVariant get(int group) {
        static constexpr int (*sizes[kMaxGroup])(int, bool) = {&smem<1>, &smem<2>, &smem<3>, &smem<4>,
                                                               &smem<5>, &smem<6>, &smem<7>, &smem<8>};
        const DecodeBuild b{reinterpret_cast<const void*>(&decode_fp4_kernel<D, BS, kWarps>), kStages, 32 * kWarps, sizes[group - 1]};
        return DecodeVariant{b, b, reinterpret_cast<const void*>(&merge_fp4_kernel<D, BS>), false, &launch};
    }
};

template <int D, int BS>
DecodeVariant pick_fp4(int group, int num_seqs, bool fixed) {
    return Fp4Layout<D, BS, 16>::bytes(group, num_seqs, fixed) <= kMaxSmem ? Fp4Variant<D, BS, 16>::get(group)
                                                                          : Fp4Variant<D, BS, 8>::get(group);
}

}  // namespace

bool decode_variant_fp4(int head_dim, int block_size, int group, int num_seqs, bool fixed, DecodeVariant* out) {
    if (head_dim == 128 && block_size == 16) *out = pick_fp4<128, 16>(group, num_seqs, fixed);
    else if (head_dim == 128 && block_size == 32) *out = pick_fp4<128, 32>(group, num_seqs, fixed);
    else if (head_dim == 64 && block_size == 16) *out = pick_fp4<64, 16>(group, num_seqs, fixed);
    else if (head_dim == 64 && block_size == 32) *out = pick_fp4<64, 32>(group, num_seqs, fixed);
    else return false;
    return true;
}

}  // namespace pa
