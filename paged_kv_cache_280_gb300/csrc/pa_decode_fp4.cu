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
//
// Measured (both kernels, device time): 256 sequences of 32 .. 4095 tokens with 32 heads of their own 165.8 us, 6.0 TB/s
// (0.89 of the measured copy rate); 4 sequences of 131072 tokens with 64 / 8 heads 100.9 us (0.89); 64 sequences with
// 32 / 8 heads 21.4 us (0.44: 4.9 us pass before a CTA's first tile arrives, 4 from its last tile to the end of the
// merge); one sequence of 1031 tokens 7.6 us.  With producer and consumer warps and four CTAs per SM, as over FP8
// pools, the first three took 299, 142 and 31 us: the hand-over cost a third of the issue slots.
#include "pa_decode.cuh"
#include "pa_decode_fp4.cuh"

namespace pa {
namespace {

// Two stages of 32 tokens a warp (2 x 4.6 KB at D = 128, 147 KB per SM): what one warp lacks in depth the
// other fifteen have.  Measured on the first two batches above (us) when it was chosen, warps x stages: 16 x 2 186 / 114,
// 14 x 2 210 / 129, 12 x 2 189 / 117, 12 x 3 192 / 118, 10 x 3 226 / 139, 8 x 4 237 / 146.  At D = 64 four stages gain nothing.
constexpr int kStageTok = 32;
constexpr size_t partial_slot_bytes_max(int d) { return (size_t)(kMaxGroup * (d + kSlotExtraFloatsPerHead) + 3) / 4 * 16; }

// What a warp has left of a segment at the end of its part: slot 0 a piece that continues a segment, slot 1 a
// segment's first piece, if the segment goes on.
struct alignas(16) Fp4Left {
    int32_t b, h;
    int32_t kind;  // 0 none; else 4, and bit 0: the segment starts in this piece, bit 1: it ends in it
    int32_t pad;
};
// kWarps: 16, one CTA per SM (512 threads of 128 registers), or 8 where a batch's prefix arrays leave no
// room for 16 rings (at D = 128 without partitions: past 2,125 sequences with 8 query
// heads to a KV head, 9,389 with one; 8 warps take 15,589 and 19,221).
template <int D, int BS, int kWarps>
struct Fp4Layout {
    static constexpr int kStages = 2;           // ring stages per warp
    static constexpr int TPS = kStageTok / BS;  // tiles per stage
    static constexpr int kTile = BS * fp4_row_bytes(D);
    static constexpr int kStageBytes = 2 * TPS * kTile;  // K of its tiles, then their V
    static constexpr int kRing = kStages * kStageBytes;  // per warp; slot 1's state goes here once the ring is idle
    static constexpr int kDescOff = kWarps * kRing;                  // int4 per stage
    static constexpr int kBarOff = kDescOff + kWarps * kStages * 16;  // full barrier per stage
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

// The plan's ranges in 32 bits, where the batch allows (`small`): the same arithmetic as Plan's without
// skew.  It comes before anything is requested from HBM, so it is worth keeping short.  Units are the plan's: weighted tiles, or partitions.
struct Fp4Ranges {
    const Plan& P;
    bool fixed, small;  // (partitions are counted in 32 bits anyhow)
    uint32_t U, C, q, r;
    // partitions: whether the plan has them; a constant where one is given
    __device__ __forceinline__ Fp4Ranges(const Plan& plan, bool partitions) : P(plan), fixed(partitions) {
        small = P.KS == 0 && P.U < (int64_t)1 << 31;
        U = (uint32_t)P.U, C = (uint32_t)P.C;
        q = U / max(C, 1u), r = U - q * C;
    }
    // the first unit of CTA c's range: c U / C = c (U / C) + c (U % C) / C, rounded up, with partitions down
    __device__ __forceinline__ uint32_t start(uint32_t c) const { return c * q + (c * r + (fixed ? 0 : C - 1)) / C; }
    // where unit x < U falls: its sequence, KV head, and the tile of the segment at or after it
    __device__ __forceinline__ void locate(uint32_t x, int32_t& b, int32_t& h, int32_t& j) const {
        const uint32_t K = Plan::K, A = P.A, H = P.Hkv;
        int lo = 0, hi = P.B - 1;  // largest sequence whose units start at or before x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((fixed ? H * P.upref[mid] : H * (K * P.pref[mid] + A * mid)) <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        const uint32_t span = fixed ? P.upref[lo + 1] - P.upref[lo] : K * P.nblocks(lo) + A;
        const uint32_t local = x - (fixed ? H * P.upref[lo] : H * (K * P.pref[lo] + A * lo));
        const uint32_t hh = local / span, rem = local - hh * span;
        b = lo, h = (int32_t)hh, j = (int32_t)(fixed ? rem * P.PT : rem <= A ? 0 : (rem - A + K - 1) / K);
    }
    __device__ __forceinline__ int32_t tile(int32_t b, int32_t h, int32_t j) const { return P.Hkv * P.pref[b] + h * P.nblocks(b) + j; }
};

// The first tile of part e (0 .. kWarps) of CTA c's range, and in seq a sequence at or before the one that
// holds it, for plans with partitions or past 32 bits.  Kept out of line: the kernel's first instructions come from
// memory, and these would lie between them.
template <int BS, int kWarps>
__device__ __noinline__ int32_t fp4_part_start_general(const DecodeParams& p, const int32_t* pref, const int32_t* upref, int c,
                                                       int e, int32_t* seq) {
    const Plan P = fp4_plan<BS>(p, pref, upref);
    if (P.PT > 0) {
        const Fp4Ranges R(P, true);
        c += e == kWarps;
        if (c == P.C) return (int32_t)P.T;
        int32_t b, h, j;
        R.locate(R.start(c), b, h, j);
        *seq = b;
        return R.tile(b, h, j);
    }
    int s0 = 0;
    int64_t split;
    const int64_t u0 = P.start_unit(c), u1 = P.start_unit(c + 1);
    const int64_t t = P.first_tile_at_unit(u0 + (u1 - u0) * e / kWarps, &split, &s0);
    *seq = s0;
    return (int32_t)t;
}
// The part (tiles t0 .. t1) of warp w of CTA c's range, and a sequence at or before the one that holds t0.
// Without partitions the parts are of equal cost in the plan's units, with partitions of equal numbers of tiles.
// The two ends are two searches, in lanes 0 and 1.
template <int BS, int kWarps>
__device__ __forceinline__ void fp4_part(const DecodeParams& p, const Plan& P, const int32_t* pref, const int32_t* upref, int c,
                                         int w, int lane, int32_t& t0, int32_t& t1, int32_t& seq) {
    const Fp4Ranges R(P, false);
    const bool fixed = P.PT > 0;
    int32_t t = 0, s = 0;
    if (P.T > 0 && c < P.C && lane < 2) {
        const int e = fixed ? kWarps * lane : w + lane;  // the end to search for; with partitions the range's own
        if (c + 1 == P.C && e == kWarps) {
            t = (int32_t)P.T;
        } else if (fixed || !R.small) {
            t = fp4_part_start_general<BS, kWarps>(p, pref, upref, c, e, &s);
        } else {
            const uint32_t u0 = R.start(c), u1 = R.start(c + 1);
            int32_t h, j;
            R.locate(u0 + (uint32_t)((uint64_t)(u1 - u0) * e / kWarps), s, h, j);
            t = R.tile(s, h, j);
        }
    }
    t0 = __shfl_sync(0xffffffffu, t, 0), t1 = __shfl_sync(0xffffffffu, t, 1);
    seq = __shfl_sync(0xffffffffu, s, 0);
    if (fixed) {
        const int32_t r0 = t0;
        const uint64_t n = (uint32_t)(t1 - t0);
        t0 = r0 + (int32_t)(n * w / kWarps), t1 = r0 + (int32_t)(n * (w + 1) / kWarps);
    }
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

// A stage's descriptor: x = valid tokens (1 .. 32) | flags | KV head << 16, y = sequence, z = stages of its piece.
enum StageFlag { kFirst = 64, kLast = 128, kStarts = 256, kEnds = 512 };

// max over the warp (no operand is a NaN).
__device__ __forceinline__ float warp_max(float x) {
    const int32_t i = __float_as_int(x), o = i ^ ((i >> 31) & 0x7fffffff);  // integers in the floats' order
    const int32_t r = __reduce_max_sync(0xffffffffu, o);
    return __int_as_float(r ^ ((r >> 31) & 0x7fffffff));
}

// One query head's sum over pieces: E elements a lane.
template <int E>
struct Fp4Sum {
    float m, l, a[E];  // m and l the same in every lane
    __device__ __forceinline__ void reset() {
        m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = 0.f;
    }
    // Adds up to 32 pieces, one to each lane in `set`, in order of the lanes: ml(lane) loads a lane's piece's (m, l)
    // for this head, at(k) is the address of lane k's piece's elements.  The loads of N pieces go together,
    // the first N with the (m, l).
    template <int N, class Ml, class At>
    __device__ __forceinline__ void add(uint32_t set, int lane, Ml ml_of, At at) {
        const bool mine = set >> lane & 1;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (mine) ml = ml_of();
        float w = 0.f;
        bool first = true;
        while (set != 0) {
            int k[N];
            float x[N][E];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                k[i] = __ffs(set) - 1;
                set &= set - 1;  // stays 0
                if (k[i] >= 0) {
                    const float* src = at(k[i]);
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 v = *reinterpret_cast<const float2*>(src + e);
                        x[i][e] = v.x, x[i][e + 1] = v.y;
                    }
                }
            }
            if (first) {
                first = false;
                const float to = fmaxf(m, warp_max(ml.x));
                const float f = to == m ? 1.f : ex2_approx(m - to);
                l *= f;
#pragma unroll
                for (int e = 0; e < E; ++e) a[e] *= f;
                m = to;
                w = !mine ? 0.f : ml.x == m ? 1.f : ex2_approx(ml.x - m);
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (k[i] >= 0) {
                    const float wk = __shfl_sync(0xffffffffu, w, k[i]);
                    l = fmaf(wk, __shfl_sync(0xffffffffu, ml.y, k[i]), l);
#pragma unroll
                    for (int e = 0; e < E; ++e) a[e] = fmaf(wk, x[i][e], a[e]);
                }
        }
    }
    __device__ __forceinline__ void store_out(__nv_bfloat16* dst, float oscale) const {
        const float r = 1.f / l;
#pragma unroll
        for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(a[e] * r * oscale, a[e + 1] * r * oscale);
    }
};

// What a CTA leaves for the merge, behind the partials: the segment of its last run, if that begins in its range and
// goes on in the next CTA's (kGoesOn; at most one does), and whether a segment that came from the one before ends
// in its range (kEndsHere).
enum Fp4RecordFlag { kGoesOn = 1, kEndsHere = 2 };
struct alignas(16) Fp4Record {
    int32_t b, h, flags, pad;
};
__device__ __forceinline__ Fp4Record* fp4_records(const DecodeParams& p, size_t slot_floats) {
    return reinterpret_cast<Fp4Record*>(p.partials + (size_t)2 * p.num_ctas * slot_floats);
}

// The lane that holds set bit number r of `set` (r < popc(set)).
__device__ __forceinline__ int nth_set_lane(uint32_t set, int r, int lane) {
    const bool is = (set >> lane & 1) && __popc(set & ((1u << lane) - 1)) == r;
    return __ffs(__ballot_sync(0xffffffffu, is)) - 1;
}

template <int D, int BS, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 1) decode_fp4_kernel(const __grid_constant__ DecodeParams p) {
    using L = Fp4Layout<D, BS, kWarps>;
    constexpr int TPS = L::TPS, NT = 32 * kWarps, kStages = L::kStages;
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
    int4* desc = reinterpret_cast<int4*>(smem + L::kDescOff) + warp * kStages;

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
    int32_t t0, t1, seq0;
    fp4_part<BS, kWarps>(p, P, pref, upref, c, warp, lane, t0, t1, seq0);

    // The walk of the copies, kStages stages ahead of the computation.  Whatever stays the same within a
    // piece or a chunk of 32 table entries is worked out when they change: a stage then costs a few
    // instructions beside its copies.
    const uint64_t policy = policy_evict_first();
    PieceIter<false> it;
    it.init(P, t0, t1, -1, seq0, seq0);
    int b = 0, j = 0, j1 = 0, rem = 0, pflags = 0;  // sequence; next tile, end tile; tokens from tile j on; flags
    int pstages = 0;                                // stages of the piece
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
        pstages = (j1 - j0 + TPS - 1) / TPS;
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
    // Copy nt tiles of the walk into ring slot s (whose previous contents this warp has read).
    auto copy = [&](int s, int nt) {
        const uint64_t o0 = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, blk, ci) * block_bytes;
        const uint64_t o1 = TPS == 1 ? 0 : (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, blk, (ci + 1) & 31) * block_bytes;
        if (elect_one()) {
            const uint32_t full = bar + 8 * s, dst = ring + s * L::kStageBytes;
            mbar_arrive_expect_tx(full, (uint32_t)(nt * 2 * L::kTile));
            bulk_load_hint(dst, kp + o0, L::kTile, full, policy);
            bulk_load_hint(dst + TPS * L::kTile, vp + o0, L::kTile, full, policy);
            if (TPS > 1 && nt > 1) {
                bulk_load_hint(dst + L::kTile, kp + o1, L::kTile, full, policy);
                bulk_load_hint(dst + (TPS + 1) * L::kTile, vp + o1, L::kTile, full, policy);
            }
        }
        ci += nt;
    };
    // The walk's next stage, any: its descriptor and copies, then the walk moves on.
    auto issue = [&](int s) {
        const int nt = TPS == 1 ? 1 : min(TPS, j1 - j);
        const bool last = j + nt == j1;
        if (lane == 0) desc[s] = make_int4(min(nt * BS, rem) | pflags | (last ? kLast : 0), b, pstages, 0);
        copy(s, nt);
        __syncwarp();
        pflags &= ~kFirst;
        j += nt;
        rem -= nt * BS;
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
    int c_left = 0;  // stages of the piece in hand that are still to be computed
    auto wait = [&]() {
        if (!__all_sync(0xffffffffu, mbar_test_wait(bar + 8 * s, parity)))
            ok = __all_sync(0xffffffffu, mbar_wait(bar + 8 * s, parity, p.wait_limit_ns));
        return ok;
    };
    while (used < issued) {
        // A run of stages inside pieces: full ones to compute, full ones to copy, no table chunk to fetch.
        int n = min(c_left, (j1 - j + TPS - 1) / TPS) - 1;
        n = have && !(pflags & kFirst) ? min(n, (32 - ci) / TPS) : 0;
        if (n >= kStages) {
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                if (!wait()) break;
                const uint32_t kb = ring + s * L::kStageBytes;
                uint32_t pb[4];
                st.template weights<false>(kb, kStageTok, lane, pb);
                st.template accumulate<false>(kb + TPS * L::kTile, kStageTok, lane, pb);
                __syncwarp();
                ++used;
                copy(s, TPS);
                ++issued;
                if (++s == kStages) s = 0, parity ^= 1;
            }
            if (!ok) break;
            if (lane < kStages) desc[lane] = make_int4(kStageTok | pflags, b, pstages, 0);  // what every slot now holds
            __syncwarp();
            c_left -= n;
            j += n * TPS;
            rem -= n * kStageTok;
            if (ci == 32) load_chunk();
        }
        // Any stage.
        const int4 d = desc[s];
        const int sh = d.x >> 16, valid = d.x & 63;
        if (d.x & kFirst) {
            st.load_q(static_cast<const __nv_bfloat16*>(p.q) + ((size_t)d.y * Hq + (size_t)sh * G) * D, G, lane, p.scale_log2);
            st.reset();
            c_left = d.z;
        }
        if (!wait()) break;
        const uint32_t kb = ring + s * L::kStageBytes, vb = kb + TPS * L::kTile;
        uint32_t pb[4];
        st.template weights<true>(kb, valid, lane, pb);
        st.template accumulate<true>(vb, valid, lane, pb);
        __syncwarp();
        ++used;
        --c_left;
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
    // Lane i looks at slot i (slot 0 of warp 0, its slot 1, slot 0 of warp 1, ...).  A run of pieces of one
    // segment opens with a slot 1, or with the CTA's first piece, and goes on through the slots 0 after it.
    // An item is one query head of one run; the warps take them in turn.
    static_assert(2 * kWarps <= 32, "a lane per slot");
    constexpr int E = D / 32;
    const Fp4Left f = left[lane & (2 * kWarps - 1)];
    const uint32_t filled = __ballot_sync(0xffffffffu, lane < 2 * kWarps && f.kind != 0);
    const uint32_t ending = __ballot_sync(0xffffffffu, lane < 2 * kWarps && (f.kind & 2));
    const uint32_t heads = filled & (0xaaaaaaaau | (filled & (0u - filled)));
    const int items = __popc(heads) * G;
    if (warp == kWarps - 1) {  // (the warp least likely to have an item)
        const int head = 31 - __clz(heads | 1u), one = __ffs(heads | 0x80000000u) - 1;  // the last run, the first
        const uint32_t later = heads & (heads - 1);                                     // the runs after the first
        const bool starts0 = __shfl_sync(0xffffffffu, f.kind, one) & 1;
        const bool ends0 = ending & (later ? (later & (0u - later)) - 1 : 0xffffffffu);
        if (lane == head)
            fp4_records(p, slot_floats)[c] = Fp4Record{f.b, f.h, (heads != 0 && (f.kind & 1) && ending >> head == 0 ? kGoesOn : 0) |
                                                                     (heads != 0 && !starts0 && ends0 ? kEndsHere : 0), 0};
    }
    auto state = [&](int slot) {
        return slot & 1 ? reinterpret_cast<const float*>(smem + (slot >> 1) * L::kRing) : slot0 + (slot >> 1) * slot_floats;
    };
    for (int item = warp; item < items; item += kWarps) {
        const int r = item / G, hq = item - r * G;
        const int head = nth_set_lane(heads, r, lane);
        const uint32_t later = heads & ~((2u << head) - 1);  // the runs after it
        const uint32_t run = filled & (0xffffffffu << head) & (later ? (later & (0u - later)) - 1 : 0xffffffffu);
        const int fb = __shfl_sync(0xffffffffu, f.b, head), fh = __shfl_sync(0xffffffffu, f.h, head);
        const int starts = __shfl_sync(0xffffffffu, f.kind, head) & 1, ends = (run & ending) ? 2 : 0;
        Fp4Sum<E> sum;
        sum.reset();
        sum.template add<4>(run, lane, [&]() { return *reinterpret_cast<const float2*>(state(lane) + G * D + 2 * hq); },
                [&](int k) { return state(k) + hq * D + E * lane; });
        if (starts && ends) {
            sum.store_out(static_cast<__nv_bfloat16*>(p.out) + ((size_t)fb * Hq + (size_t)fh * G + hq) * D + E * lane, p.out_scale);
        } else {  // slot 1: a split segment's first piece; slot 0: one that continues it
            float* dst = p.partials + (size_t)(2 * c + starts) * slot_floats;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<float2*>(dst + hq * D + E * lane + e) = make_float2(sum.a[e], sum.a[e + 1]);
            if (lane == 0) *reinterpret_cast<float2*>(dst + G * D + 2 * hq) = make_float2(sum.m, sum.l);
        }
    }
}

// The merge of split segments: M = max m_p, out = sum 2^(m_p - M) o_p / sum 2^(m_p - M) l_p over the CTAs that hold a
// piece, in an order of the kernel's own but always the same.  An item is one query head of the segment that a CTA's
// record names, if it names one.  A warp takes an item, or, where segments have four pieces or more on average, the four warps
// of a CTA share its pieces (shared / never shared: one sequence of 1031 tokens and 8 KV heads 7.6 / 8.3 us, of 4096 tokens
// and one 7.9 / 11.4; shared always, 16 sequences of 8 KV heads take 16.1 us instead of 15.1, and from two pieces on, 64 of
// one 13.5 instead of 12.5).  The decode's CTAs fill their SMs, so this kernel starts when they exit and all it does is
// latency: the records and the first pieces are fetched together, before the records say how many there are (what slots
// hold beyond them is dropped).
// Measured: its last store 2.3 us after the decode grid ends on 64 sequences of 32 / 8 heads.  When it worked the
// ranges out anew from the lengths instead of reading records, the call took 0.6 us more (21.9 us); with one CTA of 16
// warps per record 1.1 us more; merging in the decode kernel, with counters, 1.7 us less there but 5 us more on 256
// sequences of 32 heads, where its registers spilled.
constexpr int kMergeWarps = kMergeThreads / 32;
constexpr int kMergeAhead = 8;  // pieces that a warp fetches before it has the record, at most
__host__ __device__ inline bool fp4_merge_shared(int num_seqs, int num_kv_heads, int ctas) {
    return (int64_t)num_seqs * num_kv_heads * 4 <= ctas;
}
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_fp4_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int E = D / 32;
    __shared__ __align__(16) float part[kMergeWarps][D + 2];  // read two floats at a time
    static_assert((D + 2) % 2 == 0 && E % 2 == 0, "every row, and a lane's part of it, starts on 8 bytes");
    const int G = p.group, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool shared = fp4_merge_shared(p.num_seqs, p.num_kv_heads, p.num_ctas);
    const int W = shared ? kMergeWarps : 1, first = shared ? warp : 0;  // the warp takes pieces first, first + W, ...
    const int item = shared ? (int)blockIdx.x : (int)blockIdx.x * kMergeWarps + warp;
    const int ca = item / G, hq = item - ca * G;
    const size_t slot_floats = partial_slot_floats(G, D);
    // as many pieces as a segment has on average, and two
    const int guess = min(p.num_ctas / (p.num_seqs * p.num_kv_heads) + 2, min(kMergeAhead * W, p.num_ctas - ca));
    auto slot = [&](int k) { return piece_slot(p.partials, slot_floats, ca + k, ca); };
    auto ml_of = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(slot(k) + G * D) + hq); };
    auto at = [&](int k) { return slot(k) + hq * D + E * lane; };
    pdl_launch_dependents();   // what follows may start its own prologue; it waits for this grid before it reads or writes
    pdl_wait_prerequisites();  // the decode grid has finished; its records and partials are in memory
    if (ca >= p.num_ctas) return;  // (whole warps, of the last CTA, and none where warps share)
    const int4* records = reinterpret_cast<const int4*>(fp4_records(p, slot_floats));
    const int4 rec = __ldcg(records + min(ca + lane, p.num_ctas - 1));  // of the CTAs from ca on
    float2 ml[kMergeAhead];
    float x[kMergeAhead][E];
#pragma unroll
    for (int i = 0; i < kMergeAhead; ++i) {
        if (first + W * i < guess) {
            ml[i] = ml_of(first + W * i);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(at(first + W * i) + e));
                x[i][e] = v.x, x[i][e + 1] = v.y;
            }
        }
    }
    if (!(__shfl_sync(0xffffffffu, rec.z, 0) & kGoesOn)) return;
    const int b = __shfl_sync(0xffffffffu, rec.x, 0), h = __shfl_sync(0xffffffffu, rec.y, 0);
    int np = 0;  // pieces: up to the first CTA after ca in which the segment ends
    for (int from = ca, flags = lane ? rec.z : 0;;) {
        const uint32_t ends = __ballot_sync(0xffffffffu, from + lane < p.num_ctas && (flags & kEndsHere));
        np = ends ? from - ca + __ffs(ends) : p.num_ctas - ca;
        from += 32;
        if (ends != 0 || from >= p.num_ctas) break;
        flags = __ldcg(&records[min(from + lane, p.num_ctas - 1)].z);
    }
    Fp4Sum<E> sum;
    sum.reset();
#pragma unroll
    for (int i = 0; i < kMergeAhead; ++i) {
        if (first + W * i < min(np, guess)) {
            const float to = fmaxf(sum.m, ml[i].x);
            const float f = to == sum.m ? 1.f : ex2_approx(sum.m - to), w = to == ml[i].x ? 1.f : ex2_approx(ml[i].x - to);
            sum.l = fmaf(sum.l, f, w * ml[i].y);
#pragma unroll
            for (int e = 0; e < E; ++e) sum.a[e] = fmaf(sum.a[e], f, w * x[i][e]);
            sum.m = to;
        }
    }
    for (int base = guess; base < np; base += 32) {  // lane k's piece is number base + k
        const uint32_t set = __ballot_sync(0xffffffffu, base + lane < np && (base + lane) % W == first);
        sum.template add<kMergeAhead>(set, lane, [&]() { return ml_of(base + lane); }, [&](int k) { return at(base + k); });
    }
    if (shared) {
#pragma unroll
        for (int e = 0; e < E; ++e) part[warp][E * lane + e] = sum.a[e];
        if (lane == 0) part[warp][D] = sum.m, part[warp][D + 1] = sum.l;
        __syncthreads();
        if (warp != 0) return;
        sum.reset();
        sum.template add<kMergeWarps>((1u << kMergeWarps) - 1, lane, [&]() { return make_float2(part[lane][D], part[lane][D + 1]); },
                                      [&](int k) { return part[k] + E * lane; });
    }
    sum.store_out(static_cast<__nv_bfloat16*>(p.out) + ((size_t)b * p.num_q_heads + (size_t)h * G + hq) * D + E * lane,
                  p.out_scale);
}

template <int D, int BS, int kWarps>
struct Fp4Variant {
    using L = Fp4Layout<D, BS, kWarps>;
    template <int G>
    static int smem(int num_seqs, bool fixed) { return L::bytes(G, num_seqs, fixed); }
    static void launch(const DecodeParams& p, const CUtensorMap&, const CUtensorMap&, int grid, int smem_bytes, int, int,
                       cudaStream_t stream) {
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
        if (grid == 1) return;  // one CTA: nothing is split
        const unsigned items = (unsigned)grid * (unsigned)p.group;
        mcfg.gridDim = dim3(fp4_merge_shared(p.num_seqs, p.num_kv_heads, grid) ? items : (items + kMergeWarps - 1) / kMergeWarps);
        mcfg.blockDim = dim3(kMergeThreads);
        mcfg.dynamicSmemBytes = 0;
        cudaLaunchKernelEx(&mcfg, merge_fp4_kernel<D>, p);
    }
    static DecodeVariant get(int group) {
        static constexpr int (*sizes[kMaxGroup])(int, bool) = {&smem<1>, &smem<2>, &smem<3>, &smem<4>,
                                                               &smem<5>, &smem<6>, &smem<7>, &smem<8>};
        const DecodeBuild b{reinterpret_cast<const void*>(&decode_fp4_kernel<D, BS, kWarps>), L::kStages, 32 * kWarps, sizes[group - 1]};
        return DecodeVariant{b, b, reinterpret_cast<const void*>(&merge_fp4_kernel<D>), false, &launch};
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
