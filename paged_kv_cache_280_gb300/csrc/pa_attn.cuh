// Causal attention of many query rows per sequence on the fifth-generation tensor cores, over packed keys and values
// (whole prompts) or quantised pools (chunks of new tokens behind a cached context).
//
// Row i of a sequence with n new tokens at the end of len sits at position p = len - n + i and attends to the keys at
// 0 .. p:  out = softmax(scale q K^T) V,  one pass over the keys with a running maximum and sum per row.
//
// Work.  The G query heads of a KV head share its keys: for one (sequence, KV head) a tile is 128 rows, 128 / G tokens
// of G heads each, one row per TMEM lane.  A unit is two neighbouring tiles, which share every stage of 128 keys; a
// unit that holds a single tile (few new tokens) lets the tile's two TMEM halves take the even and the odd stages
// instead, so that either way one half's softmax runs while the tensor core works for the other.
//   Packed: the units, most keys first, are dealt to the CTAs in snake order (PackedWalk).
//   Pools:  the units' stages are laid end to end and cut in equal parts (pa_attn_plan.h), so that few rows over a long
//           context fill the card; the pieces of cut units are joined by a second kernel (attn_join_kernel).
//
// Warps.  0 .. 3 and 4 .. 7: the softmax of the two halves, a thread per row.  8: keys and values.  9 and 10: the MMAs
// of the two halves.  11: the walk over the work (AttnPieces), and query rows (packed).  12 .. 15 (pools): query rows and
// widening of the codes.
//   Packed: K and V stages by TMA, 128-byte swizzle, a ring of slots in shared memory.
//   Pools:  the blocks' codes by bulk copies into a ring of raw slots; the widening warps turn them into f16 (exact for
//           E4M3, and for E2M1 codes times their E4M3 scale) in the swizzled layout, with zeros for rows behind the
//           sequence's end.  Query rows are scaled by a power of two and rounded to f16 on the way.
//   S = Q K^T into TMEM (M 128, N 128), O += P V with P read from TMEM, where the softmax wrote it over S's last 64 columns.
//   P is handed over in two halves of 64 keys, so that the product with V begins while the second half's exponentials
//   are formed.
// O is rescaled in TMEM only when a row's maximum has grown by more than 2^8 since it was last scaled.  Scores too large for a
// weight's exponent to be one fma leave the loop for one of their own (at_softmax_large).  Every wait is
// bounded; one that gives up sets PA_DEV_WAIT_TIMEOUT, every role stops, and the CTA waits for its own copies and MMAs
// before it frees TMEM.
//
// Bound and measured.  Two 128 x 128 x 128 products a stage and tile are 1024 cycles of the tensor core; Q and K of an S, both
// from shared memory, take all its 128 bytes a clock meanwhile.  The softmax of a stage is some 1900 cycles of a half's warps
// (128 exponentials a thread, TMEM both ways), which the other half's products cover but for its hand-overs, so a stage of
// two tiles takes about 3500 (the products' 2050).  A unit's end and the next one's start cost some 3000 more.
//   Packed, 64 / 8 heads of 128: one prompt of 8191 tokens 792 to 838 us from one card to the next, 1.31 to 1.39 PFLOP/s (0.69 to
//   0.73 of the measured bf16 rate; tensor pipe busy 59 %); 32 / 8 heads: 16 prompts of 1031 tokens 160 us (0.46: a unit has five
//   stages on average, the last one masked).
//   Pools: the widening beside it (4 warps, about 1100 cycles of conversions and stores for K or V of a stage, which share the
//   issue slots and shared memory with the rest).  4-bit, 32 / 8 heads of 128, 2047 tokens at the end of 32767: 848 us (0.66); 2 x 9
//   tokens over 131072 keys, 64 / 8 heads: 134 us (tiles of 72 rows and less are padded to 128, so the tensor core's 44 % busy
//   cycles and the widening bound it, not HBM's 45 us); FP8, 32 / 32 heads, 129 to 517 tokens over up to 16383 keys: 158 us (HBM
//   57; a tile is one head's, so every key is widened for 256 rows at most).
#pragma once

#include <atomic>
#include <cmath>
#include <type_traits>

#include "pa_attn_plan.h"
#include "pa_device.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

enum AttnSource { kAttnPacked = 0, kAttnFp8 = 1, kAttnFp4 = 2 };

struct AttnParams {
    void* out;
    const uint16_t* q;             // pools: bf16 [tokens][Hq][D]; packed: through the tensor maps
    const uint8_t *k_pool, *v_pool;
    const int32_t* block_tables;
    const int32_t* seq_lens;       // null: packed
    const int32_t* cu_q_lens;
    int32_t* status;
    int4* cuts;                    // pools: [grid] the cut unit that begins in a CTA: first row of q, tokens, KV head, last CTA (-1: none)
    float2* part_ml;               // pools: [2 * grid slots][tiles][128]: reference (base 2, times kAtRefUnit) and sum of a row's piece
    float* part_o;                 // pools: [2 * grid slots][tiles][128][D]
    int32_t part_tiles;            // tiles per slot
    int32_t max_blocks_per_seq, num_seqs, num_q_heads, num_kv_heads, num_blocks, num_q_tokens, max_q_len, bs_shift;
    int32_t group, tile_tokens;    // G, 128 / G rounded down
    uint32_t group_inverse;        // 2^16 / G rounded up: rows below 256 divided by G
    int32_t out_align32;           // out is 32-byte aligned: 32-byte stores
    int32_t max_len;               // pools: the longest context that a table holds (kAttnMaxLen at most)
    float scale_log2, out_scale;   // pools: scale_log2 in [1, 2], times 2^scale_exp
    int32_t scale_exp;
    int32_t wait_limit_ns;         // kWaitLimitNs, or less in tests
};
static_assert(kWaitLimitNs <= INT32_MAX, "a wait's limit is handed to the kernel in 32 bits");

constexpr int kAtRows = 128;
constexpr int kAtKvWarp = 8, kAtMmaWarp = 9, kAtQWarp = 11, kAtWidenWarp = 12;
constexpr uint32_t kAtTmemCols = 512;  // half t: S (P over its last 64 columns) in 256 t + [0, 128), O in 256 t + 128 + [0, D)
constexpr uint32_t kAtTmemHalf = 256;
constexpr uint32_t kAtTmemP = 64, kAtTmemO = 128;
constexpr float kAtRescaleLog2 = 8.f;
// f16 weights are held times 2^7: with the lazy rescaling they stay below 2^15 (2^15.25 where their shift is coarse), and keep
// all their bits down to 2^-21 of the largest.
constexpr float kAtWeightLog2 = 7.f;
// A weight is 2^(c s + shift), one fma, with shift = 7 - c m (packed: -c m) rounded to fp32, the same for all keys that share
// m; what rescales and joins takes differences of such shifts, so their rounding cancels.  It is 1 / 4 at most, and the f16
// weights stay in range, while |c m| is below this; a piece with larger scores goes to at_softmax_large.
constexpr float kAtLargeLog2 = 4194304.f;
// A piece's reference (minus its shift) is handed on times this: finite however large c m is.
constexpr float kAtRefUnit = 1.f / 4294967296.f;

template <int I = 0, int N, class F>
__device__ __forceinline__ void at_static_for_impl(F& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        at_static_for_impl<I + 1, N>(f);
    }
}
template <int N, class F>  // f(integral_constant<int, i>) for i = 0 .. N - 1
__device__ __forceinline__ void at_static_for(F&& f) {
    at_static_for_impl<0, N>(f);
}

// 2^x on the SFU (ex2.approx: 2^-22 relative); 2^-inf = +0.
__device__ __forceinline__ float at_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The shift of a row whose maximum is m: rounded once, the same way wherever it is formed.
template <int SRC>
__device__ __forceinline__ float at_shift(float m, float c) {
    return __fmaf_rn(-m, c, SRC == kAttnPacked ? 0.f : kAtWeightLog2);
}
// 2^x, x a difference of references.
__device__ __forceinline__ float at_ref_exp2(float x) { return at_exp2(x * (1.f / kAtRefUnit)); }

template <int SRC, int D>
struct AttnLayout {
    static constexpr bool kPools = SRC != kAttnPacked;
    static constexpr int kThreads = kPools ? 512 : 384;
    // Registers a thread: at launch (all that a CTA alone on its SM can have), and the warpgroups' shares of those: two of
    // softmax, loads and MMA, widening.
    static constexpr int kRegs = 65536 / kThreads / 8 * 8;
    static constexpr int kSoftmaxRegs = kPools ? 168 : 216, kLoadRegs = kPools ? 80 : 72, kWidenRegs = kPools ? 96 : 0;
    static_assert(2 * kSoftmaxRegs + kLoadRegs + kWidenRegs <= kThreads / 128 * kRegs, "more registers than the launch has: a wait for ever");
    static constexpr int kPanels = D / 64;
    static constexpr int kPanelBytes = 128 * 128;           // 128 rows (query rows or keys) of 64 elements
    static constexpr int kTileBytes = kPanels * kPanelBytes;  // a query tile, or K or V of a stage
    static constexpr int kSlots = kPools ? (D == 128 ? 3 : 5) : (D == 128 ? 5 : 8);
    static constexpr int kRawBytes = SRC == kAttnFp8 ? 128 * D : 128 * fp4_row_bytes(D);
    static constexpr int kRaws = !kPools ? 0 : SRC == kAttnFp8 ? 4 : D == 128 ? 6 : 8;  // even: a slot always serves the same pair of widening warps
    static constexpr int kRingOff = 2 * kTileBytes;
    static constexpr int kRawOff = kRingOff + kSlots * kTileBytes;
    static constexpr int kRowOff = kRawOff + kRaws * kRawBytes;  // pools: row factors' exponents [2 pieces][2 tiles][128] bytes
    static constexpr int kMlOff = kRowOff + (kPools ? 2 * 2 * 128 : 0);  // odd half's maximum and sum (below 0: a large piece's) [128]
    static constexpr int kBarOff = kMlOff + 128 * 8;
    static constexpr int kNumBars = 2 * kSlots + 2 * kRaws + 21;
    static constexpr int kMiscOff = (kBarOff + kNumBars * 8 + 15) / 16 * 16;  // abort flag, limit, TMEM address; work range at + 16
    static constexpr int kPieceOff = kMiscOff + 80;                           // two pieces of kPieceBytes
    static constexpr int kPieceBytes = 48;
    static constexpr int kBytes = kPieceOff + 2 * kPieceBytes + 1024;  // +1 KB to align the base
    static_assert(kBytes <= kMaxSmem, "shared memory");
};

template <int SRC, int D>
struct AttnBars {
    using L = AttnLayout<SRC, D>;
    uint32_t base;
    __device__ uint32_t at(int i) const { return base + 8u * i; }
    __device__ uint32_t full(int s) const { return at(s); }
    __device__ uint32_t empty(int s) const { return at(L::kSlots + s); }
    __device__ uint32_t raw_full(int s) const { return at(2 * L::kSlots + s); }
    __device__ uint32_t raw_empty(int s) const { return at(2 * L::kSlots + L::kRaws + s); }
    static constexpr int kRest = 2 * L::kSlots + 2 * L::kRaws;
    __device__ uint32_t s_full(int t) const { return at(kRest + t); }        // S in TMEM
    __device__ uint32_t p_first(int t) const { return at(kRest + 2 + t); }   // weights of keys 64 .. 127 in TMEM, O rescaled
    __device__ uint32_t p_second(int t) const { return at(kRest + 4 + t); }  // the other weights
    __device__ uint32_t o_final(int t) const { return at(kRest + 6 + t); }   // a piece's last P V
    __device__ uint32_t q_full() const { return at(kRest + 8); }
    __device__ uint32_t q_empty() const { return at(kRest + 9); }
    __device__ uint32_t tail() const { return at(kRest + 10); }      // packed: a V box with rows behind its sequence's end
    __device__ uint32_t odd_ml() const { return at(kRest + 11); }    // the odd half's maximum and sum are in shared memory
    __device__ uint32_t odd_read() const { return at(kRest + 12); }  // the even half's warps have read them, and its O
    __device__ uint32_t drain(int t) const { return at(kRest + 13 + t); }
    __device__ uint32_t piece_full(int i) const { return at(kRest + 17 + i); }   // a piece's entry is written
    __device__ uint32_t piece_empty(int i) const { return at(kRest + 19 + i); }  // every warp of a role has read it
    __device__ uint32_t turn(int t) const { return at(kRest + 15 + t); }  // the half's turn at the tensor core
};

// One thread's wait, for `limits` times the launch's limit (behind the abort flag) at most; gives up once that flag is set.  (The flag and the clock are looked at now and
// then only: a thread that is busy with them notices late that its phase has completed.)
__device__ __forceinline__ bool at_wait1(uint32_t bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* status,
                                         uint32_t limits = 1) {
    uint64_t since = 0;
    for (int n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n & 31) continue;
        if (*abort_flag) return false;
        const uint64_t now = global_timer_ns();
        if (since == 0) {
            since = now;
        } else if (now - since > (uint64_t)(uint32_t)abort_flag[1] * limits) {
            *abort_flag = 1;
            flag_status(status, PA_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
    return true;
}
// The same for a warp: its lanes go on together.
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity, volatile int32_t* abort_flag, int32_t* status,
                                        uint32_t limits = 1) {
    return __all_sync(0xffffffffu, at_wait1(bar, parity, abort_flag, status, limits));
}
// For the waits that last as long as a piece: one of the longest context that fits into memory takes some 20 s.  (Where a
// copy or an MMA is lost, the other roles notice within one limit.)
constexpr uint32_t kPieceLimits = 32;

__device__ __forceinline__ int at_token(const AttnParams& p, int row) { return (int)((uint32_t)row * p.group_inverse >> 16); }

// ---- work ------------------------------------------------------------------------------------------

// New tokens of sequence b (0: none, or a sequence that breaks the call's bounds), its first row and its length.
template <int SRC>
__device__ __forceinline__ int at_sequence(const AttnParams& p, int b, int& c0, int& len, bool* bad = nullptr) {
    c0 = __ldg(p.cu_q_lens + b);
    len = SRC == kAttnPacked ? INT32_MAX : __ldg(p.seq_lens + b);
    bool wrong;
    const int n = sequence_tokens(c0, __ldg(p.cu_q_lens + b + 1), len, p.num_q_tokens, p.max_q_len,
                                  SRC == kAttnPacked ? INT32_MAX : p.max_len, wrong);
    if (SRC == kAttnPacked) len = n;
    if (bad) *bad = wrong;
    return n;
}

// A run of stages of one unit.  All roles take the same pieces in the same order.
struct AttnPiece {
    int b, g, c0, n, len;
    int i0;         // the unit's first new token
    bool one;       // a single tile, whose halves take the even and the odd stages
    int k0, ns;     // stages k0 .. k0 + ns - 1 of the unit
    int n0;         // two tiles: how many of them the first tile sees
    bool first, last;  // the unit's first, last stage is among them
    int cut_end;    // pools: the last CTA of a cut unit that begins here, else -1
    int nst;        // the unit's stages (of the walks)
};

__device__ __forceinline__ void at_fields(const AttnParams& p, int m, AttnPiece& w) {
    const int T = p.tile_tokens;
    w.i0 = 2 * m * T;
    w.one = w.i0 + T >= w.n;
    const int base = w.len - w.n;
    w.nst = (base + min(w.n, w.i0 + 2 * T) + kAttnKeys - 1) / kAttnKeys;
}
__device__ __forceinline__ void at_stages(const AttnParams& p, int k0, int k1, AttnPiece& w) {
    w.k0 = k0, w.ns = k1 - k0;
    const int nst0 = (w.len - w.n + min(w.n, w.i0 + p.tile_tokens) + kAttnKeys - 1) / kAttnKeys;
    w.n0 = max(0, min(k1, nst0) - k0);
    w.first = k0 == 0, w.last = k1 == w.nst;
}

// Packed: the units that exist, 256 sequences at a time, in them by unit index from the last down (the most keys first), then
// sequence, then KV head; CTA c takes ranks c, 2 C - 1 - c, 2 C + c, ..  Every unit index looked at has units among the 256
// sequences, so that the walk is no longer than eight steps a unit and eight for each 256 sequences, however loose the bound on
// the lengths is.  The walk counts from step to step (`off`), so that no number of units leaves 32 bits.  Warp-collective.
struct PackedWalk {
    static constexpr int kTogether = 256;
    int first, m, chunk, loaded, mine;
    int off;  // from the first unit of this step (unit index, 32 sequences) to the CTA's next
    bool back;  // the snake goes backwards there
    uint32_t mask;
    __device__ PackedWalk() : first(-kTogether), m(-1), chunk(0), loaded(-1), mine(0), off(blockIdx.x), back(false), mask(0) {}
    __device__ __forceinline__ void load(const AttnParams& p) {  // how many units the chunk's 32 sequences have
        if (loaded == chunk) return;
        const int b = chunk + (threadIdx.x & 31);
        int c0, len;
        const int n = b < p.num_seqs ? at_sequence<kAttnPacked>(p, b, c0, len) : 0;
        mine = (n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
        loaded = chunk;
    }
    __device__ __forceinline__ int end(const AttnParams& p) const { return min(first + kTogether, p.num_seqs); }
    __device__ __forceinline__ void begin(const AttnParams& p) {  // at the 256 sequences from `first` on
        int most = 0;
        for (chunk = first; chunk < end(p); chunk += 32) load(p), most = max(most, mine);
        m = (int)__reduce_max_sync(0xffffffffu, (unsigned)most) - 1;
        chunk = first;
        load(p);
        mask = __ballot_sync(0xffffffffu, mine > m);
    }
    __device__ __forceinline__ bool next(const AttnParams& p, AttnPiece& w) {
        while (first < p.num_seqs) {
            if (m < 0) {
                first += kTogether;
                begin(p);
                continue;
            }
            const int here = __popc(mask) * p.num_kv_heads;
            if (off < here) {
                const int j = off / p.num_kv_heads;
                w.g = off - j * p.num_kv_heads;
                w.b = chunk + __fns(mask, 0, j + 1);
                w.n = at_sequence<kAttnPacked>(p, w.b, w.c0, w.len);
                at_fields(p, m, w);
                at_stages(p, 0, w.nst, w);
                w.cut_end = -1;
                off += 2 * (back ? (int)blockIdx.x : (int)(gridDim.x - 1 - blockIdx.x)) + 1;
                back = !back;
                return true;
            }
            off -= here;
            chunk += 32;
            if (chunk >= end(p)) chunk = first, --m;
            load(p);
            mask = __ballot_sync(0xffffffffu, mine > m);
        }
        return false;
    }
};

// Pools: this CTA's range of the line of work (written by at_plan before the roles start).
struct AttnRange {
    int64_t at, end, W;  // the first unit's beginning, the range's end; the whole line
    int32_t b, g, m, k, C, U;
    int32_t n, len, c0;  // of sequence b
};
struct RangeWalk {
    int64_t at, end, W;
    int b, g, m, k, U, C;
    bool fresh;
    int n, len, c0;
    __device__ RangeWalk(const AttnParams&, const void* range) : fresh(false) {
        const volatile AttnRange* r = static_cast<const volatile AttnRange*>(range);
        at = r->at, end = r->end, b = r->b, g = r->g, m = r->m, k = r->k, n = r->n, len = r->len, c0 = r->c0, U = r->U;
        W = r->W, C = r->C;
    }
    __device__ __forceinline__ bool next(const AttnParams& p, AttnPiece& w) {
        while (at < end) {
            if (fresh) {
                n = at_sequence<kAttnFp8>(p, b, c0, len);
                fresh = false;
                if (n == 0) {  // (some later sequence has tokens: the range has not ended)
                    ++b, fresh = true;
                    continue;
                }
            }
            w.b = b, w.g = g, w.n = n, w.len = len, w.c0 = c0;
            at_fields(p, m, w);
            const int wt = w.one ? kOneTile : kTwoTiles;
            const int k0 = min(k, w.nst), k1 = (int)min((int64_t)w.nst, stage_at(end - at, wt, U));
            w.cut_end = k0 == 0 && k1 < w.nst ? (int)range_of(at + stage_begin(w.nst - 1, wt, U), W, C) : -1;
            if (k1 < w.nst) {
                at = end;
            } else {
                at += (w.one ? U / 2 : U) + (int64_t)(len - n + min(n, w.i0 + 2 * p.tile_tokens)) * wt;
                k = 0;
                if (2 * ++m * p.tile_tokens >= n) {
                    m = 0;
                    if (++g == p.num_kv_heads) g = 0, ++b, fresh = true;
                }
            }
            if (k0 < k1) {
                at_stages(p, k0, k1, w);
                return true;
            }
        }
        return false;
    }
};

// One warp: this CTA's range.
__device__ __forceinline__ void at_plan(const AttnParams& p, AttnRange* range, int lane) {
    int c0_mine = 0, U = 0;
    auto line = [&](int b) {
        int c0 = 0, len = 0;
        const int n = b < p.num_seqs ? at_sequence<kAttnFp8>(p, b, c0, len) : 0;
        c0_mine = c0;
        return UnitLine{n, len, p.tile_tokens, U};
    };
    int64_t W = 0, W1 = 0;  // with U = 0, and with 2, which takes it twice for a unit of two tiles and once for one of one
    UnitLine mine_line{};
    for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
        mine_line = line(b0 + lane);
        W += mine_line.total() * p.num_kv_heads;
        mine_line.U = 2;
        W1 += mine_line.total() * p.num_kv_heads;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o), W1 += __shfl_xor_sync(0xffffffffu, W1, o);
    const int64_t units = W1 - W;
    U = unit_weight(W, units, gridDim.x, p.part_tiles == 1);
    W += units * (U / 2);
    const int64_t C = W > 0 ? ranges(W, gridDim.x, U, p.part_tiles == 1) : 0, c = blockIdx.x;
    if (c >= C) {
        if (lane == 0) range->at = range->end = 0, range->W = W, range->C = (int)C;
        return;
    }
    const int64_t x = range_begin(c, W, C);
    int64_t before = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
        if (p.num_seqs > 32) mine_line = line(b0 + lane);
        mine_line.U = U;
        const int64_t mine = mine_line.total() * p.num_kv_heads;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int64_t lo = before + incl - mine;
        if (lo <= x && x < before + incl) {
            const UnitLine u = mine_line;
            const int64_t per_head = u.total();
            int64_t r = x - lo;
            const int g = (int)(r / per_head);
            r -= g * per_head;
            const int m = u.unit_at(r);
            r -= u.before(m);
            range->b = b0 + lane, range->g = g, range->m = m, range->n = u.n, range->len = u.len, range->c0 = c0_mine;
            range->k = (int)min(stage_at(r, u.key_weight(m), U), (int64_t)INT32_MAX), range->U = U;
            range->at = x - r, range->end = range_begin(c + 1, W, C), range->W = W, range->C = (int)C;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// Sequences that break the call's bounds are flagged by one warp of the first CTA, when it has nothing else to do.
template <int SRC>
__device__ __forceinline__ void at_flag_sequences(const AttnParams& p, int lane) {
    if (blockIdx.x) return;
    for (int b = lane; b < p.num_seqs; b += 32) {
        int c0, len;
        bool bad;
        at_sequence<SRC>(p, b, c0, len, &bad);
        if (bad) flag_status(p.status, PA_DEV_BAD_SEQ_LEN);
    }
}

// The pieces in shared memory: one warp walks and writes them two ahead, the other roles read them.  (Walked by every role
// for itself, the MMA and softmax warps' walk, about 2000 cycles, lay between a piece's last stage and the next one's first.)
template <int SRC, int D>
struct AttnPieces {
    using L = AttnLayout<SRC, D>;
    uint8_t* base;
    AttnBars<SRC, D> bars;
    int i;
    __device__ AttnPieces(uint8_t* base, const AttnBars<SRC, D>& bars) : base(base), bars(bars), i(0) {}
    __device__ __forceinline__ void get(int n, AttnPiece& w) const {
        const uint32_t at = bars.base - L::kBarOff + L::kPieceOff + (n & 1) * L::kPieceBytes;
        const uint4 a = lds16(at), b = lds16(at + 16), c = lds16(at + 32);
        const int4 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w}, y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w}, z = {(int)c.x, (int)c.y, (int)c.z, 0};
        w.b = x.x, w.g = x.y, w.c0 = x.z, w.n = x.w;
        w.len = y.x, w.i0 = y.y, w.k0 = y.z, w.ns = y.w;
        w.n0 = z.x, w.one = z.y & 1, w.first = z.y & 2, w.last = z.y & 4, w.cut_end = z.z, w.nst = 0;
    }
    // A whole warp: the next piece; false behind the last one, or when a wait has been given up.
    __device__ __forceinline__ bool next(AttnPiece& w, volatile int32_t* abort_flag, int32_t* status, int lane) {
        if (!at_wait(bars.piece_full(i & 1), (i >> 1) & 1, abort_flag, status)) return false;
        get(i, w);
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.piece_empty(i & 1));
        ++i;
        __syncwarp();
        return w.ns > 0;
    }
    // The same for one thread that reads alone for its warp.
    __device__ __forceinline__ bool next1(AttnPiece& w, volatile int32_t* abort_flag, int32_t* status) {
        if (!at_wait1(bars.piece_full(i & 1), (i >> 1) & 1, abort_flag, status)) return false;
        get(i, w);
        mbar_arrive(bars.piece_empty(i & 1));
        ++i;
        return w.ns > 0;
    }
    // The walking warp: piece i (have: false behind the last one).
    __device__ __forceinline__ bool put(const AttnPiece& w, bool have, volatile int32_t* abort_flag, int32_t* status, int lane) {
        if (!at_wait(bars.piece_empty(i & 1), ((i >> 1) & 1) ^ 1, abort_flag, status, kPieceLimits)) return false;
        if (lane == 0) {
            int4* e = reinterpret_cast<int4*>(base + L::kPieceOff + (i & 1) * L::kPieceBytes);
            e[0] = make_int4(w.b, w.g, w.c0, w.n);
            e[1] = make_int4(w.len, w.i0, w.k0, have ? w.ns : 0);
            e[2] = make_int4(w.n0, (w.one ? 1 : 0) | (w.first ? 2 : 0) | (w.last ? 4 : 0), w.cut_end, 0);
            mbar_arrive(bars.piece_full(i & 1));
        }
        ++i;
        __syncwarp();
        return true;
    }
};

// The stages of a piece in the order of their slots: K runs ahead of V by one stage, by two where two halves of one
// tile take turns.
struct AttnItems {
    int k, v, ns, lead;
    __device__ AttnItems(const AttnPiece& w) : k(0), v(0), ns(w.ns), lead(w.one ? 2 : 1) {}
    __device__ __forceinline__ bool next(int& stage) {  // true: V
        if (k < ns && k < v + lead) {
            stage = k++;
            return false;
        }
        stage = v++;
        return true;
    }
};

// The stage of a piece's item i in that order (keys are zeroed behind the sequence's end like values: nothing reads them).
__device__ __forceinline__ int at_item_stage(const AttnPiece& w, int i) {
    if (!w.one) return i >> 1;
    const int first = min(2, w.ns), m = i - first;  // the keys ahead, then a stage's values and the keys two on
    return m < 0 ? i : m < 2 * (w.ns - first) ? (m >> 1) + ((m & 1) << 1) : i - w.ns;
}

// The slots of a piece's stages in that order, from the first slot c on.
struct AttnSlots {
    int c, ns, lead;
    __device__ AttnSlots(const AttnPiece& w, int c) : c(c), ns(w.ns), lead(w.one ? 2 : 1) {}
    __device__ __forceinline__ int k(int j) const { return c + (lead == 1 ? 2 * j : j < 2 ? j : 2 * j - 1); }
    __device__ __forceinline__ int v(int j) const { return c + (lead == 1 ? 2 * j + 1 : min(2 * j + 2, ns + j)); }
};

template <int NS>
struct AttnRing {  // a slot of NS and the parity of its fill
    uint32_t slot, parity;
    __device__ __forceinline__ void ahead(uint32_t by) {  // by < 2 NS
        slot += by;
        if (slot >= NS) slot -= NS, parity ^= 1u;
        if (slot >= NS) slot -= NS, parity ^= 1u;
    }
};

// ---- loads -----------------------------------------------------------------------------------------

// Packed: K and V of each stage, a box of 128 tokens per 64-element panel.  The stage that reaches past its sequence
// holds rows of the next one, or anything: its V rows there are zeroed (a weight of zero times NaN is NaN) before the
// slot counts as full, so its box lands on a barrier that only this warp waits for.
template <int D>
__device__ __forceinline__ void at_load_packed(const AttnParams& p, const CUtensorMap* tk, const CUtensorMap* tv, uint8_t* base,
                                               uint32_t base_s, const AttnBars<kAttnPacked, D>& bars,
                                               volatile int32_t* abort_flag, int lane) {
    using L = AttnLayout<kAttnPacked, D>;
    if (lane == 0) {
        prefetch_tensormap(tk);
        prefetch_tensormap(tv);
    }
    AttnPieces<kAttnPacked, D> pieces(base, bars);
    AttnPiece w;
    int sc = 0, tails = 0;
    bool ok = true;
    while (ok && pieces.next(w, abort_flag, p.status, lane)) {
        AttnItems items(w);
        for (int i = 0; i < 2 * w.ns; ++i, ++sc) {
            int j;
            const bool is_v = items.next(j);
            const int s = sc % L::kSlots;
            if (!at_wait(bars.empty(s), ((sc / L::kSlots) & 1) ^ 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            const int key0 = (w.k0 + j) * kAttnKeys;
            const uint32_t dst = L::kRingOff + s * L::kTileBytes;
            const bool tail = is_v && key0 + kAttnKeys > w.len;
            const uint32_t bar = tail ? bars.tail() : bars.full(s);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, (uint32_t)L::kTileBytes);
#pragma unroll
                for (int pn = 0; pn < L::kPanels; ++pn)
                    tma_load_3d(base_s + dst + pn * L::kPanelBytes, is_v ? tv : tk, pn * 64, w.g, w.c0 + key0, bar);
            }
            __syncwarp();
            if (tail) {
                if (!at_wait(bar, tails & 1, abort_flag, p.status)) {
                    mbar_wait(bar, tails & 1);  // (the box must land before the CTA ends)
                    ok = false;
                    break;
                }
                ++tails;
                const int z0 = w.len - key0, nz = (kAttnKeys - z0) * 8;  // rows, then 16-byte chunks of a panel
                for (int e = lane; e < nz * L::kPanels; e += 32) {
                    const int pn = e >= nz ? 1 : 0, rem = e - pn * nz;
                    *reinterpret_cast<uint4*>(base + dst + pn * L::kPanelBytes + z0 * 128 + rem * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.full(s));
            }
        }
    }
    // never leave the CTA with copies still landing in its shared memory
    for (int kk = sc > L::kSlots ? sc - L::kSlots : 0; kk < sc; ++kk) mbar_wait(bars.full(kk % L::kSlots), (kk / L::kSlots) & 1);
}

// Packed: a piece's query tiles (3-D boxes of 64 elements x G heads x 128 / G tokens), once the last piece's Q K^T have
// completed.  A warp of its own, so that keys and values run ahead into the next piece; it also walks.
template <int D>
__device__ __forceinline__ void at_load_q_packed(const AttnParams& p, const CUtensorMap* tq, uint8_t* base, uint32_t base_s,
                                                 const AttnBars<kAttnPacked, D>& bars, volatile int32_t* abort_flag, int lane) {
    using L = AttnLayout<kAttnPacked, D>;
    if (lane == 0) prefetch_tensormap(tq);
    const uint32_t tile_bytes = (uint32_t)(L::kPanels * p.group * p.tile_tokens * 128);
    PackedWalk walk;
    AttnPieces<kAttnPacked, D> pieces(base, bars);
    AttnPiece ahead, w;
    int pc = 0;
    bool more = true;  // pieces to put
    auto put = [&]() {
        const bool have = walk.next(p, ahead);
        more = pieces.put(ahead, have, abort_flag, p.status, lane) && have;
    };
    put();
    if (more) put();
    for (;;) {
        if (pc == pieces.i) break;  // (a wait was given up)
        pieces.get(pc, w);
        if (w.ns == 0) break;
        if (!at_wait(bars.q_empty(), (pc & 1) ^ 1, abort_flag, p.status, kPieceLimits)) break;
        if (lane == 0) {
            const int tiles = w.one ? 1 : 2;
            mbar_arrive_expect_tx(bars.q_full(), tile_bytes * tiles);
            for (int t = 0; t < tiles; ++t)
#pragma unroll
                for (int pn = 0; pn < L::kPanels; ++pn)
                    tma_load_3d(base_s + t * L::kTileBytes + pn * L::kPanelBytes, tq, pn * 64, w.g * p.group,
                                w.c0 + w.i0 + t * p.tile_tokens, bars.q_full());
        }
        __syncwarp();
        ++pc;
        if (more) put();
    }
    if (pc > 0) mbar_wait(bars.q_full(), (pc - 1) & 1);
    __syncwarp();
    at_flag_sequences<kAttnPacked>(p, lane);
    __syncwarp();
}

// Pools: the walk, a warp of its own.
template <int SRC, int D>
__device__ __forceinline__ void at_walk(const AttnParams& p, AttnRange* range, uint8_t* base, const AttnBars<SRC, D>& bars,
                                        volatile int32_t* abort_flag, int lane) {
    at_plan(p, range, lane);
    __syncwarp();
    RangeWalk walk(p, range);
    AttnPieces<SRC, D> pieces(base, bars);
    AttnPiece w;
    for (bool more = true; more;) {
        const bool have = walk.next(p, w);
        more = pieces.put(w, have, abort_flag, p.status, lane) && have;
    }
    __syncwarp();
    at_flag_sequences<SRC>(p, lane);
    __syncwarp();
}

// Pools: the codes of each stage's blocks, one bulk copy a block (its rows of one KV head are contiguous).  The table
// entry of the next item is fetched before the wait for a free slot.
template <int SRC, int D>
__device__ __forceinline__ void at_load_raw(const AttnParams& p, uint8_t* base, uint32_t base_s, const AttnBars<SRC, D>& bars,
                                            volatile int32_t* abort_flag, int lane) {
    using L = AttnLayout<SRC, D>;
    const int per = kAttnKeys >> p.bs_shift;                       // blocks per stage
    const uint32_t bytes = (uint32_t)(L::kRawBytes / kAttnKeys) << p.bs_shift;  // of a block and head
    AttnPieces<SRC, D> pieces(base, bars);
    AttnPiece w;
    int sc = 0;
    bool ok = true;
    while (ok && pieces.next(w, abort_flag, p.status, lane)) {
        const int blocks = (w.len + (1 << p.bs_shift) - 1) >> p.bs_shift;
        const int32_t* table = p.block_tables + (int64_t)w.b * p.max_blocks_per_seq;
        AttnItems items(w);
        int j, j_next = 0;
        bool is_v, v_next = items.next(j_next);
        auto entry = [&](int stage) {
            const int e = (w.k0 + stage) * per + lane;
            return lane < per && e < blocks ? __ldg(table + e) : 0;
        };
        int32_t id_next = entry(j_next);
        for (int i = 0; i < 2 * w.ns; ++i, ++sc) {
            j = j_next, is_v = v_next;
            int32_t id = id_next;
            if (i + 1 < 2 * w.ns) {
                v_next = items.next(j_next);
                id_next = entry(j_next);
            }
            const int s = sc % L::kRaws;
            if (!at_wait(bars.raw_empty(s), ((sc / L::kRaws) & 1) ^ 1, abort_flag, p.status)) {
                ok = false;
                break;
            }
            const int have = min(per, blocks - (w.k0 + j) * per);
            if (lane == 0) mbar_arrive_expect_tx(bars.raw_full(s), bytes * have);
            __syncwarp();
            if (lane < have) {
                if (id < 0 || id >= p.num_blocks) {
                    flag_status(p.status, PA_DEV_BAD_BLOCK_ID);
                    id = 0;
                }
                bulk_load(base_s + L::kRawOff + s * L::kRawBytes + lane * bytes,
                          (is_v ? p.v_pool : p.k_pool) + ((int64_t)id * p.num_kv_heads + w.g) * bytes, bytes, bars.raw_full(s));
            }
            __syncwarp();
        }
    }
    for (int kk = sc > L::kRaws ? sc - L::kRaws : 0; kk < sc; ++kk) mbar_wait(bars.raw_full(kk % L::kRaws), (kk / L::kRaws) & 1);
}

__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Pools: a piece's query rows as f16, each scaled by a power of two so that its largest element lies in [1, 2), and the
// inverse factors.  Warp `part` of four takes every fourth group of rows.  The rows are copied to where they belong as
// they are, all at once, and then rewritten there, each chunk by the lane that copied it.  Rows of no token stay as they
// are: they reach no other row.
template <int SRC, int D>
struct AttnQueries {
    using L = AttnLayout<SRC, D>;
    static constexpr int kLanes = D / 8, kRowsAt = 32 / kLanes;  // lanes per row, rows at a time
    int rows, tile_rows, r0, c;
    uint32_t base_s;
    const uint16_t* src;
    __device__ AttnQueries(const AttnParams& p, const AttnPiece& w, uint32_t base_s, int part, int lane) : base_s(base_s) {
        c = lane % kLanes, r0 = part * kRowsAt + lane / kLanes;
        tile_rows = p.tile_tokens * p.group;
        rows = min(w.n - w.i0, w.one ? p.tile_tokens : 2 * p.tile_tokens) * p.group;
        src = p.q + ((int64_t)(w.c0 + w.i0) * p.num_q_heads + w.g * p.group) * D + c * 8;
    }
    __device__ __forceinline__ uint32_t chunk(int at) const {
        const int t = at >= tile_rows ? 1 : 0, r = at - t * tile_rows;
        return base_s + t * L::kTileBytes + (c >> 3) * L::kPanelBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
    __device__ __forceinline__ void copy(const AttnParams& p) const {
#pragma unroll 2
        for (int at = r0; at < rows; at += 4 * kRowsAt) {
            const int tok = at_token(p, at);
            copy_ahead16(chunk(at), src + ((int64_t)tok * p.num_q_heads + (at - tok * p.group)) * D);
        }
        copies_commit();
    }
    __device__ __forceinline__ void widen(uint8_t* factors) const {
        copies_wait<0>();
#pragma unroll 2
        for (int at0 = r0 - r0 % kRowsAt; at0 < rows; at0 += 4 * kRowsAt) {  // (the same turns for every lane: rows meet in shuffles)
            const int at = at0 + r0 % kRowsAt;
            const uint32_t here = chunk(min(at, rows - 1));
            const uint4 x = lds16(here);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
            uint32_t top = 0;  // largest magnitude, as bf16 bits
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, xs[e] & 0x7fff7fffu);
#pragma unroll
            for (int o = 1; o < kLanes; o *= 2) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t e2 = min(max(max(top & 0xffffu, top >> 16) >> 7, 1u), 253u);  // its exponent
            const float inv = __uint_as_float((254u - e2) << 23);
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = pack_f16x2(bf16_lo(xs[e]) * inv, bf16_hi(xs[e]) * inv);
            if (at < rows) {
                sts16(here, h[0], h[1], h[2], h[3]);
                if (c == 0) factors[at >= tile_rows ? 128 + at - tile_rows : at] = (uint8_t)e2;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
    }
};

// Pools: raw codes to f16 in the swizzled layout (128-byte rows of 64 elements, 16-byte chunk c of row r at c ^ (r & 7)).
// Two of the four warps (numbers `part`) take an item (K or V of a stage), the other two the next, a warp 64 rows.  In each
// group of eight lanes the rows and chunks are chosen so that neither the loads nor the stores meet in a bank:
//   FP8: two rows, four 16-byte chunks (16 codes) of each, the first half of one row and the second of the other;
//   4-bit: four rows, two 16-byte chunks (32 codes, two scales) of each; at head_dim 128 two rows' first halves and two
//   rows' second halves.
// How far the loop is unrolled weighs its latencies against the instruction cache, which all roles share (32 sequences of 5
// tokens, FP8, and 2 of 9 over 131072 4-bit keys: 2 turns 113 and 164 us, 4: 112 and 139, all: 125 and 142).  All four warps
// on each item wait for each item's barriers: 127 and 156.
template <int SRC, int D>
__device__ __forceinline__ void at_widen(const AttnParams& p, uint8_t* base, uint32_t base_s, const AttnBars<SRC, D>& bars,
                                         volatile int32_t* abort_flag, int part, int lane) {
    using L = AttnLayout<SRC, D>;
    constexpr int kRows = kAttnKeys / 2;  // of a warp and item
    constexpr int kPerRow = D == 128 ? 2 : 1;        // turns per row: the other half of the row
    constexpr int kStep = SRC == kAttnFp8 ? 8 : 16;  // rows a turn (of two)
    constexpr int kTurns = kRows / kStep * kPerRow;
    AttnPieces<SRC, D> pieces(base, bars);
    AttnPiece w;
    int pc = 0;
    // the pair's first raw slot and slot
    AttnRing<L::kRaws> raws{(uint32_t)part >> 1, 0u};
    AttnRing<L::kSlots> slots{(uint32_t)part >> 1, 0u};
    const int l8 = lane & 7, l4 = lane >> 3;
    const int r_first = kRows * (part & 1) + (SRC == kAttnFp8 ? 2 * l4 + (l8 >> 2) : 4 * l4 + (l8 >> 1));
    const uint32_t panel_first = D == 128 ? l8 >> 2 : 0;
    const uint32_t r7 = (uint32_t)r_first & 7u;
    // where the thread's first codes and scales are in a raw slot; 4-bit: from 16 rows to the next 16, and on to those behind
    // them (a block's record: its rows' codes, then their scales)
    const uint32_t rec = (uint32_t)(L::kRawBytes / kAttnKeys) << p.bs_shift, off = (uint32_t)r_first & ((1u << p.bs_shift) - 1u);
    const uint32_t codes_at = SRC == kAttnFp8 ? r_first * 128 + (l8 & 3) * 16
                                              : ((uint32_t)r_first >> p.bs_shift) * rec + off * (D / 2) + (l8 & 1) * 16;
    const uint32_t scales_at = ((uint32_t)r_first >> p.bs_shift) * rec + ((D / 2) << p.bs_shift) + off * (D / 16) + (l8 & 1) * 2;
    const uint32_t codes_16 = p.bs_shift == 4 ? rec : 16 * (D / 2), scales_16 = p.bs_shift == 4 ? rec : 16 * (D / 16);
    const uint32_t codes_32 = p.bs_shift == 4 ? 2 * rec : rec;
    struct Codes {
        uint4 c;
        uint16_t scales;
    };
    while (pieces.next(w, abort_flag, p.status, lane)) {
        // The query rows first if their place is free already; else the first keys are widened before it is.
        const AttnQueries<SRC, D> queries(p, w, base_s, part, lane);
        const uint32_t q_parity = (pc & 1) ^ 1;
        const bool q_free = __all_sync(0xffffffffu, mbar_test_wait(bars.q_empty(), q_parity));
        auto load_queries = [&]() {
            queries.copy(p);
            queries.widen(base + L::kRowOff + (pc & 1) * 256);
            if (lane == 0) mbar_arrive(bars.q_full());
        };
        if (q_free) load_queries();
        bool q_due = !q_free;
        for (int i = part >> 1; i < 2 * w.ns; i += 2) {  // (a piece's items are even in number)
            if (q_due && i > 0) {
                q_due = false;
                if (!at_wait(bars.q_empty(), q_parity, abort_flag, p.status)) return;
                load_queries();
            }
            if (!at_wait(bars.raw_full(raws.slot), raws.parity, abort_flag, p.status)) return;
            const uint32_t raw = base_s + L::kRawOff + raws.slot * L::kRawBytes;
            auto load = [&](int turn) {
                const uint32_t step = turn / kPerRow, panel = panel_first ^ (turn & (kPerRow - 1));
                Codes x;
                if constexpr (SRC == kAttnFp8) {
                    x.c = lds16(raw + codes_at + step * (kStep * 128) + panel * 64);
                    x.scales = 0;
                } else {
                    const uint32_t there = raw + (step >> 1) * codes_32;
                    x.c = lds16(there + codes_at + (step & 1) * codes_16 + panel * 32);
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x.scales) : "r"(there + scales_at + (step & 1) * scales_16 + panel * 4) : "memory");
                }
                return x;
            };
            Codes next = load(0);
            const uint32_t dst = base_s + L::kRingOff + slots.slot * L::kTileBytes;
            const int keep = min(kAttnKeys, w.len - (w.k0 + at_item_stage(w, i)) * kAttnKeys);  // rows of the sequence
            if (!at_wait(bars.empty(slots.slot), slots.parity ^ 1u, abort_flag, p.status)) return;
#pragma unroll 4
            for (int turn = 0; turn < kTurns; ++turn) {
                Codes x = next;
                if (turn + 1 < kTurns) next = load(turn + 1);
                const int r = r_first + turn / kPerRow * kStep;
                const uint32_t row = dst + (panel_first ^ (turn & (kPerRow - 1))) * L::kPanelBytes + r * 128;
                if constexpr (SRC == kAttnFp8) {
                    const uint32_t ch = 2 * (l8 & 3);
                    uint32_t h[8];
                    e4m3x4_to_f16x2(x.c.x, h[0], h[1]);
                    e4m3x4_to_f16x2(x.c.y, h[2], h[3]);
                    e4m3x4_to_f16x2(x.c.z, h[4], h[5]);
                    e4m3x4_to_f16x2(x.c.w, h[6], h[7]);
                    sts16(row + ((ch ^ r7) << 4), h[0], h[1], h[2], h[3]);
                    sts16(row + (((ch + 1) ^ r7) << 4), h[4], h[5], h[6], h[7]);
                } else {
                    const uint32_t sc2 = e4m3x2_to_f16x2(x.scales), s0 = f16x2_low_twice(sc2), s1 = f16x2_high_twice(sc2);
                    const uint32_t xs[4] = {x.c.x, x.c.y, x.c.z, x.c.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t h[4];
                        e2m1x8_to_f16x2(xs[e], h);
#pragma unroll
                        for (int f = 0; f < 4; ++f) h[f] = mul_f16x2(h[f], e < 2 ? s0 : s1);
                        sts16(row + (((4 * (l8 & 1) + e) ^ r7) << 4), h[0], h[1], h[2], h[3]);
                    }
                }
            }
            if (keep < kAttnKeys) {  // (the whole warp) rows behind the sequence's end: whatever is there may be NaN
#pragma unroll 1
                for (int turn = 0; turn < kTurns; ++turn) {
                    const int r = r_first + turn / kPerRow * kStep;
                    const uint32_t row = dst + (panel_first ^ (turn & (kPerRow - 1))) * L::kPanelBytes + r * 128;
                    const int first = SRC == kAttnFp8 ? 2 * (l8 & 3) : 4 * (l8 & 1);
                    if (r < keep) continue;
#pragma unroll 1
                    for (int e = first; e < first + (SRC == kAttnFp8 ? 2 : 4); ++e) sts16(row + ((e ^ r7) << 4), 0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                // Only now is the raw slot free: its codes were in registers long ago, but nothing orders a shared-memory
                // load that has not returned before the next copy into the slot, only the use of what it loaded does.
                mbar_arrive(bars.raw_empty(raws.slot));
                mbar_arrive(bars.full(slots.slot));
            }
            raws.ahead(2), slots.ahead(2);
        }
        if (q_due) {
            if (!at_wait(bars.q_empty(), q_parity, abort_flag, p.status)) return;
            load_queries();
        }
        ++pc;
    }
}

// ---- MMA -------------------------------------------------------------------------------------------
// One thread issues each half's MMAs (P V of a stage, then S of its next), and the two take turns: an MMA holds up its
// issuer until the tensor core takes it, so whatever else that thread does (waits, addresses, fetching code that the
// softmax has pushed out of the instruction cache: about 600 cycles a turn, beside 1024 of MMAs) must run beside the other
// thread's MMAs.  Without turns the halves fall into step and wait for the tensor core, and it for them, at once.
template <int SRC, int D>
__device__ __forceinline__ void at_mma(const AttnParams& p, uint32_t t, uint8_t* base, uint32_t base_s, uint32_t tmem,
                                       const AttnBars<SRC, D>& bars, volatile int32_t* abort_flag, int lane) {
    using L = AttnLayout<SRC, D>;
    constexpr int NS = L::kSlots;
    constexpr int kBf16 = SRC == kAttnPacked ? 1 : 0;
    constexpr uint32_t idesc_s = umma_idesc_16(kAtRows, kAttnKeys, 0, 0, kBf16);  // Q (K-major) x K^T (K-major)
    constexpr uint32_t idesc_o = umma_idesc_16(kAtRows, D, 0, 1, kBf16);          // P (TMEM) x V (MN-major)
    const uint32_t q_lo = (uint32_t)umma_smem_desc(base_s, 16, 1024);
    const uint32_t k_lo = (uint32_t)umma_smem_desc(base_s + L::kRingOff, 16, 1024);
    const uint32_t v_lo = (uint32_t)umma_smem_desc(base_s + L::kRingOff, L::kPanelBytes, 1024);
    constexpr uint32_t hi = (uint32_t)(umma_smem_desc(0, 0, 1024) >> 32);
    constexpr uint32_t kTile16 = L::kTileBytes >> 4, kPanel16 = L::kPanelBytes >> 4;
    // S (at d) = Q K^T over half of the head's elements, 16 at a time: 32 bytes along a 128-byte row, 64-element panels
    // further apart
    auto issue_s = [&](uint32_t d, uint32_t qa, uint32_t kb, auto h_c) {
        at_static_for<D / 32>([&](auto ks_c) {
            constexpr int ks = D / 32 * decltype(h_c)::value + decltype(ks_c)::value;
            constexpr uint32_t o = (ks >> 2) * kPanel16 + (ks & 3) * 2;
            umma_bf16_lo<o, o>(d, qa, kb, hi, idesc_s, ks > 0 ? 1u : 0u);
        });
    };
    // O (behind S) += P V over keys 64 h .. 64 h + 63 of the stage, 16 keys (16 rows of 128 bytes) at a time
    auto issue_o = [&](uint32_t d, uint32_t vb, auto h_c, uint32_t acc0) {
        constexpr int h = decltype(h_c)::value;
        at_static_for<4>([&](auto i_c) {
            constexpr int i = decltype(i_c)::value, kk = 4 * h + i;
            umma_bf16_tmem_a_lo<kk * 128>(d + kAtTmemO, d + kAtTmemP + kk * 8, vb, hi, idesc_o, i > 0 ? 1u : acc0);
        });
    };
    using Ring = AttnRing<NS>;
    AttnPieces<SRC, D> pieces(base, bars);
    AttnPiece w;
    Ring first{0u, 0u};           // the piece's first slot
    uint32_t pc = 0, ck = 0, rounds = 0;  // pieces, stages of this half, turns
    const uint32_t d = tmem + kAtTmemHalf * t;
    // One lane all the way, and the next piece's entry read ahead: what it does between a piece's last MMA and the next
    // one's first is what the tensor core waits for (with the warp meeting at each piece 3000 cycles).
    if (lane == 0) {
        AttnPiece ahead;
        bool ok = true, more = pieces.next1(w, abort_flag, p.status), given = false;  // given: the piece's first S is issued
        while (ok && more) {
            using First = std::integral_constant<int, 0>;
            using Second = std::integral_constant<int, 1>;
            // In round r the half has its turn: P V of stage j, S of stage j + lead.  Of two tiles both see every stage, of
            // one tile half 0 has the even stages and half 1 the odd ones.
            const AttnSlots at(w, 0);
            const int lead = at.lead, n = w.one || t ? w.ns : w.n0, last = w.one ? (w.ns - 1) / 2 : w.ns - 1;
            const uint32_t qa = q_lo + (w.one ? 0u : t * kTile16);
            int j = (w.one ? (int)t : 0) - lead;
            Ring kr = first, vr = first;
            if (w.one && t) kr.ahead(at.k(1));
            vr.ahead(at.v(j + lead));
            // A half without a stage does not wait for the queries: it has no say in when they are replaced, so it could find
            // the barrier two phases on.  (Its turns tell it that they were there.)
            if (!given && j + lead < n) ok = at_wait1(bars.q_full(), pc & 1, abort_flag, p.status);
            bool early = false;
#pragma unroll 1
            for (int r = -1; ok && r <= last; ++r) {
                if (r == last) more = pieces.next1(ahead, abort_flag, p.status);
                const bool product = j >= 0 && j < n;
                bool scores = j + lead < n && !(given && r < 0);
                Ring ks = kr;
                bool k_alone = w.one || j + lead >= w.n0, q_vote = j + 2 * lead >= n, q_alone = w.one ? w.ns == 1 : w.n0 == 0;
                // Packed: the first half's last turn is empty where its tile does not see the unit's last stage.  Then the next
                // piece's first S takes it, as soon as its queries are there (for which the other half has done its part: its
                // last S of this piece has been issued), and runs beside the other half's last softmax (16 prompts of 1031
                // tokens: 158 us, without it 165).  Over pools, where the queries come later, the turn is better passed on
                // (162 us against 157 on the FP8 turns).
                if (SRC == kAttnPacked && r == last && !product && t == 0 && more && (ahead.one || ahead.n0 > 0)) {
                    early = scores = true;
                    ks = first;
                    ks.ahead((uint32_t)(2 * w.ns) % (2 * NS));
                    k_alone = ahead.one, q_vote = ahead.one ? ahead.ns <= 2 : ahead.n0 == 1, q_alone = ahead.one && ahead.ns == 1;
                }
                const uint32_t vb = v_lo + vr.slot * kTile16, kb = k_lo + ks.slot * kTile16;
                if (product) ok = at_wait1(bars.full(vr.slot), vr.parity, abort_flag, p.status) &&
                                  at_wait1(bars.p_first(t), ck & 1, abort_flag, p.status);
                ok = ok && at_wait1(bars.turn(t), (rounds & 1) ^ (t ^ 1), abort_flag, p.status);
                if (ok && early && r == last) ok = at_wait1(bars.q_full(), (pc + 1) & 1, abort_flag, p.status);
                if (!ok) break;
                const bool k_over = scores && mbar_test_wait(bars.full(ks.slot), ks.parity);
                // A slot is released by both halves: a half that is alone with a stage gives the other's vote at once.
                auto release = [&](uint32_t bar, bool alone) {
                    if (alone) mbar_arrive(bar);
                    umma_commit(bar);
                };
                if (product) {
                    tc_fence_after();
                    const bool over = mbar_test_wait(bars.p_second(t), ck & 1);
                    issue_o(d, vb, Second{}, j < lead ? 0u : 1u);
                    if (!over && !at_wait1(bars.p_second(t), ck & 1, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_o(d, vb, First{}, 1u);
                    release(bars.empty(vr.slot), w.one || j >= w.n0);
                    ++ck;
                }
                if (scores) {
                    if (!k_over && !at_wait1(bars.full(ks.slot), ks.parity, abort_flag, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_s(d, qa, kb, First{});
                }
                mbar_arrive(bars.turn(t ^ 1));  // (the other's first MMA comes behind the rest of these)
                if (scores) {
                    issue_s(d, qa, kb, Second{});
                    umma_commit(bars.s_full(t));
                    release(bars.empty(ks.slot), k_alone);
                    if (q_vote) release(bars.q_empty(), q_alone);  // the half's last S
                } else if (product) {
                    umma_commit(bars.o_final(t));
                }
                ++rounds;
                if (j >= 0) vr.ahead(at.v(j + lead) - at.v(j));
                kr.ahead(at.k(j + 2 * lead) - at.k(j + lead));
                j += lead;
            }
            first.ahead((uint32_t)(2 * w.ns) % (2 * NS));
            ++pc;
            w = ahead, given = early;
        }
    }
    __syncwarp();
    // every MMA issued has completed before the CTA may free TMEM or its shared memory
    if (lane == 0) {
        umma_commit(bars.drain(t));
        mbar_wait(bars.drain(t), 0);
    }
    __syncwarp();
}

// ---- softmax ---------------------------------------------------------------------------------------

// 32 fp32 values as 32 bf16 at dst.
__device__ __forceinline__ void at_store_bf16(uint16_t* dst, const float* x, bool align32) {
    uint32_t v[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
    if (align32) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * e), "r"(v[8 * e]),
                         "r"(v[8 * e + 1]), "r"(v[8 * e + 2]), "r"(v[8 * e + 3]), "r"(v[8 * e + 4]), "r"(v[8 * e + 5]),
                         "r"(v[8 * e + 6]), "r"(v[8 * e + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(dst)[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    }
}

// The rest of a piece, from stage i on (whose scores have arrived), for a warp some of whose rows have scores past
// kAtLargeLog2: their maximum is taken off the scores before c scales them, P = 2^(c (s - m)) (pools: 2^7 of it), at any size.
// Apart from the loop below, whose registers and code it leaves alone (with a branch for such rows in it, all others took 2 to
// 10 % longer): each stage's scores pass through twice, quarter by quarter.
template <int SRC, int D>
__device__ __forceinline__ bool at_softmax_large(const AttnBars<SRC, D>& bars, int t, volatile int32_t* abort_flag, int32_t* status,
                                                 uint32_t row_tmem, float c, const AttnPiece& w, int pos, int pos_high, int lane,
                                                 int i, int mine, int& ck, float& m_raw, float& l_run) {
    constexpr float kTop = SRC == kAttnPacked ? 0.f : kAtWeightLog2;
    // what the loop before has summed is relative to its rounded shift
    const float old_shift = at_shift<SRC>(m_raw, c);
    const int i0 = i;
#pragma unroll 1
    for (; i < mine; ++i, ++ck) {
        if (i > i0 && !at_wait(bars.s_full(t), ck & 1, abort_flag, status)) return false;
        tc_fence_after();
        __syncwarp();
        const int key0 = (w.k0 + (w.one ? 2 * i + t : i)) * kAttnKeys;
        const int nq = max(0, min(4, (pos_high - key0 + 32) >> 5));
        uint32_t x[32];
        auto load = [&](int q) {
            const int seen = pos - key0 - 32 * q;
            tmem_ld32(row_tmem + 32 * q, x);
            tmem_wait_ld32(x);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e > seen) x[e] = __float_as_uint(-INFINITY);
        };
        float m_new = m_raw;
#pragma unroll 1
        for (int q = 0; q < nq; ++q) {
            load(q);
#pragma unroll
            for (int e = 0; e < 32; ++e) m_new = fmaxf(m_new, __uint_as_float(x[e]));
        }
        if (i > 0) {
            const float f = m_raw == -INFINITY ? 0.f
                            : i == i0          ? at_exp2(kTop - fmaf(m_new, c, old_shift))
                                               : at_exp2((m_raw - m_new) * c);
            if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                for (int c0o = 0; c0o < D; c0o += 32) {
                    tmem_ld32(row_tmem + kAtTmemO + c0o, x);
                    tmem_wait_ld32(x);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                    tmem_st32(row_tmem + kAtTmemO + c0o, x);
                }
                l_run *= f;
            }
        }
        m_raw = m_new;
        const float less = m_raw > -INFINITY ? m_raw : 0.f;
#pragma unroll 1
        for (int q = 3; q >= 0; --q) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) pw[e] = 0u;
            if (q < nq) {
                load(q);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float x0 = at_exp2(fmaf(__uint_as_float(x[e]) - less, c, kTop));
                    const float x1 = at_exp2(fmaf(__uint_as_float(x[e + 1]) - less, c, kTop));
                    l_run += x0 + x1;
                    pw[e / 2] = SRC == kAttnPacked ? pack_bf16x2(x0, x1) : pack_f16x2(x0, x1);
                }
            }
            tmem_st16(row_tmem + kAtTmemP + 16 * q, pw);
            if (q & 1) continue;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q ? bars.p_first(t) : bars.p_second(t));
            __syncwarp();
        }
    }
    return true;
}

// Half t: warps 4 t .. 4 t + 3, row r = 32 (warp % 4) + lane = TMEM lane r.
template <int SRC, int D>
__device__ __forceinline__ void at_softmax(const AttnParams& p, int t, uint8_t* base, uint32_t tmem,
                                           const AttnBars<SRC, D>& bars, volatile int32_t* misc, int warp, int lane) {
    using L = AttnLayout<SRC, D>;
    constexpr float kTop = SRC == kAttnPacked ? 0.f : kAtWeightLog2;
    volatile int32_t* abort_flag = misc;
    const int G = p.group, Hq = p.num_q_heads, T = p.tile_tokens;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16), row_tmem = lanes + kAtTmemHalf * t;
    float2* odd_ml = reinterpret_cast<float2*>(base + L::kMlOff);
    float c = p.scale_log2;  // > 0 (checked on the host); pools: the row's, below
    int ck = 0, pc = 0, oc0 = 0, oc1 = 0, hand = 0;  // stages, pieces, final O of each half, odd halves handed over
    AttnPieces<SRC, D> pieces(base, bars);
    AttnPiece w;
    while (pieces.next(w, abort_flag, p.status, lane)) {
        const int mine = w.one ? (t ? w.ns / 2 : (w.ns + 1) / 2) : (t ? w.ns : w.n0);
        const bool other = w.one && w.ns > 1;  // both halves work on the one tile
        const int tile = w.one ? 0 : t;
        const int i0 = w.i0 + tile * T, i1 = min(w.n, i0 + T);
        const int tok = i0 + at_token(p, r);
        const bool valid = r < T * G && tok < i1;
        const int pos = w.len - w.n + (valid ? tok : i1 - 1);
        const int pos_low = __shfl_sync(0xffffffffu, pos, 0), pos_high = __shfl_sync(0xffffffffu, pos, 31);  // (they do not fall)
        float m_raw = -INFINITY, l_run = 0.f;  // maximum of the raw scores, and the weights' sum
        auto shift_of = [&](float m) { return at_shift<SRC>(m, c); };
        // (of the warp's rows; those of no token hold anything and have no say)
        auto is_large = [&](float m) { return __any_sync(0xffffffffu, valid && m > -INFINITY && fabsf(m) * c > kAtLargeLog2) != 0; };
        int i = 0;
        for (; i < mine; ++i, ++ck) {
            const int k = w.k0 + (w.one ? 2 * i + t : i);
            if (!at_wait(bars.s_full(t), ck & 1, abort_flag, p.status)) return;
            tc_fence_after();
            if constexpr (SRC != kAttnPacked) {  // (the factors were written before the MMAs of this S were issued)
                if (i == 0) {
                    // The row's factor goes through c's exponent, held inside fp32's: a c of 0 or infinity would make NaN of a
                    // masked or a zero score.  Where it is held, nothing changes: S is below 2^21, so at 2^-126 all the row's
                    // weights are 1, and unequal scores differ by 2^-34 and more, so at 2^126 all but the largest's are 0.
                    const int e = reinterpret_cast<const volatile uint8_t*>(base + L::kRowOff)[(pc & 1) * 256 + tile * 128 + r];
                    c = p.scale_log2 * __uint_as_float((uint32_t)min(max((valid ? e : 127) + p.scale_exp, 1), 253) << 23);
                }
            }
            __syncwarp();  // (TMEM instructions want the whole warp, here and wherever lanes part before one)
            // This S was issued after the last P V of this half and completes after it: O is up to date, and no MMA
            // touches this half's TMEM until this warp arrives on p_first.
            const int key0 = k * kAttnKeys;
            const int nq = min(4, (pos_high - key0 + 32) >> 5);  // quarters that some row of the warp sees
            // Masked scores become -inf: the quarters that reach past the position of some of the warp's rows are rewritten so
            // first, those past all of them (from nq on) without being read.  (With those left out of the maximum instead, the
            // branches cost every stage more: one prompt of 8191 tokens 838 us against 827, 2 x 9 tokens over 131072 keys 143
            // against 133.)
            if (key0 + kAttnKeys - 1 > pos_low) {
#pragma unroll 1
                for (int q = max(0, pos_low + 1 - key0) >> 5; q < 4; ++q) {
                    uint32_t x[32];
                    const int seen = pos - key0 - 32 * q;
                    if (q < nq) {
                        tmem_ld32(row_tmem + 32 * q, x);
                        tmem_wait_ld32(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e > seen) x[e] = __float_as_uint(-INFINITY);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(-INFINITY);
                    }
                    tmem_st32(row_tmem + 32 * q, x);
                }
                tmem_wait_st();
            }
            // The stage's 128 scores of this row pass through twice, for the maximum and for the weights, with the last two
            // quarters kept and the first two read again (all of them at once would take 128 registers).  Quarter by
            // quarter from the last to the first, the weights go over S's last 64 columns, behind those still to be read.
            // (The loops stay rolled for the instruction cache.)
            uint32_t xa[32], xb[32], xc[32];
            float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
            auto larger = [&](const uint32_t(&x)[32]) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    mx0 = fmax3(mx0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    mx1 = fmax3(mx1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                    mx2 = fmax3(mx2, __uint_as_float(x[e + 4]), __uint_as_float(x[e + 5]));
                    mx3 = fmax3(mx3, __uint_as_float(x[e + 6]), __uint_as_float(x[e + 7]));
                }
            };
            tmem_ld32(row_tmem, xc);
            tmem_ld32(row_tmem + 32, xa);
            tmem_wait_ld32(xc);
            tmem_wait_ld32(xa);
            tmem_ld32(row_tmem + 96, xb);
            larger(xc);
            tmem_ld32(row_tmem + 64, xc);
            larger(xa);
            tmem_wait_ld32(xb);
            tmem_wait_ld32(xc);
            larger(xb);
            larger(xc);
            const float m_new = fmaxf(m_raw, fmaxf(fmax3(mx0, mx1, mx2), mx3));
            if (i == 0) {
                if (is_large(m_new)) break;
                m_raw = m_new;
            } else {
                const bool need = (m_new - m_raw) * c > kAtRescaleLog2;
                if (__any_sync(0xffffffffu, need)) {
                    if (is_large(m_new)) break;
                    const float f = need ? at_exp2(shift_of(m_new) - shift_of(m_raw)) : 1.f;
#pragma unroll 1
                    for (int c0o = 0; c0o < D; c0o += 32) {
                        uint32_t x[32];
                        tmem_ld32(row_tmem + kAtTmemO + c0o, x);
                        tmem_wait_ld32(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                        tmem_st32(row_tmem + kAtTmemO + c0o, x);
                    }
                    l_run *= f;
                    m_raw = need ? m_new : m_raw;
                }
            }
            // P = 2^(c s - c m) (over pools 2^7 of it).  A row that has seen no key yet weighs all of them 0.
            const float shift = shift_of(m_raw > -INFINITY ? m_raw : 0.f);
            const uint64_t c2 = f2_pack(c, c), sh2 = f2_pack(shift, shift);
            uint64_t sum2 = f2_pack(0.f, 0.f);
            auto weigh = [&](int q, const uint32_t(&x)[32]) {
                uint32_t pw[16];
                if (q >= nq) {  // past the warp's last position
#pragma unroll
                    for (int e = 0; e < 16; ++e) pw[e] = 0u;
                } else {
                    // exponents of four pairs ahead of the exponentials of the four before them
                    uint64_t y[4];
#pragma unroll
                    for (int e = 0; e < 20; ++e) {
                        if (e >= 4) {
                            float x0, x1;
                            f2_unpack(y[e & 3], x0, x1);
                            x0 = at_exp2(x0);
                            x1 = at_exp2(x1);
                            sum2 = f2_add(sum2, f2_pack(x0, x1));
                            pw[e - 4] = SRC == kAttnPacked ? pack_bf16x2(x0, x1) : pack_f16x2(x0, x1);
                        }
                        if (e < 16)
                            y[e & 3] = f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, sh2);
                    }
                }
                tmem_st16(row_tmem + kAtTmemP + 16 * q, pw);
            };
#pragma unroll 1
            for (int h = 1; h >= 0; --h) {
                weigh(2 * h + 1, xb);
                if (h) tmem_ld32(row_tmem + 32, xb);
                weigh(2 * h, xc);
                if (h) tmem_ld32(row_tmem, xc);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(h ? bars.p_first(t) : bars.p_second(t));
                __syncwarp();
                if (h) {
                    tmem_wait_ld32(xb);
                    tmem_wait_ld32(xc);
                }
            }
            float sa, sb;
            f2_unpack(sum2, sa, sb);
            l_run += sa + sb;
        }
        bool large = i < mine;  // of the warp's rows: O and l_run are relative to 2^(c m - kTop), not to 2^-shift
        if (large && !at_softmax_large<SRC, D>(bars, t, abort_flag, p.status, row_tmem, c, w, pos, pos_high, lane, i, mine, ck, m_raw, l_run))
            return;
        ++pc;
        if (w.one && t == 1) {
            if (mine > 0) {
                odd_ml[r] = make_float2(m_raw, large ? -l_run : l_run);
                __syncwarp();
                if (lane == 0) mbar_arrive(bars.odd_ml());
                if (!at_wait(bars.odd_read(), hand & 1, abort_flag, p.status)) return;
                ++hand, ++oc1;
            }
            continue;
        }
        // ---- O / l to out, or O, m and l to the join ----
        const bool whole = w.first && w.last;
        float f0 = 1.f, f1 = 0.f;
        if (mine > 0) {
            int& oc = t ? oc1 : oc0;
            if (!at_wait(bars.o_final(t), oc & 1, abort_flag, p.status)) return;
            ++oc;
        }
        if (t == 0 && !w.one) ++oc1;
        if (other) {
            if (!at_wait(bars.o_final(1), oc1 & 1, abort_flag, p.status)) return;
            if (!at_wait(bars.odd_ml(), hand & 1, abort_flag, p.status)) return;
            ++oc1, ++hand;
            const float2 o = odd_ml[r];
            const float top = fmaxf(m_raw, o.x);
            const bool odd_large = o.y < 0.f, any_large = large || odd_large;
            auto factor = [&](float m, bool was_large) {  // from a half's reference to both halves'
                const float x = !any_large ? shift_of(top) - shift_of(m) : was_large ? (m - top) * c : kTop - fmaf(top, c, shift_of(m));
                return m > -INFINITY ? at_exp2(x) : 0.f;
            };
            f0 = factor(m_raw, large), f1 = factor(o.x, odd_large);
            l_run = l_run * f0 + fabsf(o.y) * f1;
            m_raw = top, large = any_large;
        }
        __syncwarp();
        tc_fence_after();
        const int64_t row = ((int64_t)(w.c0 + (valid ? tok : i0)) * Hq + (int64_t)w.g * G + (r - (tok - i0) * G)) * D;
        const int64_t part = SRC == kAttnPacked ? 0 : ((int64_t)(2 * blockIdx.x + (w.first ? 1 : 0)) * p.part_tiles + tile) * kAtRows + r;
        if (mine > 0) {
            const float inv = whole ? p.out_scale / l_run : 1.f;
            f0 *= inv, f1 *= inv;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t ov[32];
                float x[32];
                tmem_ld32(row_tmem + kAtTmemO + 32 * q, ov);
                tmem_wait_ld32(ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(ov[e]) * f0;
                if (other) {
                    tmem_ld32(lanes + kAtTmemHalf + kAtTmemO + 32 * q, ov);
                    tmem_wait_ld32(ov);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] += __uint_as_float(ov[e]) * f1;
                }
                if (valid && whole) {
                    at_store_bf16(static_cast<uint16_t*>(p.out) + row + 32 * q, x, p.out_align32);
                } else if constexpr (SRC != kAttnPacked) {
                    if (valid) {
                        const float* dst = p.part_o + part * D + 32 * q;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            asm volatile("st.global.cg.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + e), "f"(x[e]),
                                         "f"(x[e + 1]), "f"(x[e + 2]), "f"(x[e + 3]), "f"(x[e + 4]), "f"(x[e + 5]), "f"(x[e + 6]),
                                         "f"(x[e + 7])
                                         : "memory");
                    }
                }
                __syncwarp();
            }
        }
        tc_fence_before();  // the O reads are ordered before this warp's next arrival
        if (other) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bars.odd_read());
        }
        if constexpr (SRC != kAttnPacked) {
            if (!whole && valid) {
                const float ref = large ? m_raw * (c * kAtRefUnit) - kTop * kAtRefUnit : -shift_of(m_raw) * kAtRefUnit;
                __stcg(p.part_ml + part, make_float2(m_raw > -INFINITY ? ref : -INFINITY, l_run));
            }
            if (w.cut_end >= 0 && t == 0 && r == 0)
                p.cuts[blockIdx.x] = make_int4(w.c0 + i0, min(w.n - i0, w.one ? T : 2 * T), w.g, w.cut_end);
        }
    }
}

// ---- kernel ----------------------------------------------------------------------------------------
template <int SRC, int D>
__global__ void __launch_bounds__(AttnLayout<SRC, D>::kThreads, 1)
    attn_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v) {
    using L = AttnLayout<SRC, D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw), base_s = (raw_s + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_s - raw_s);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int32_t* misc = reinterpret_cast<volatile int32_t*>(base + L::kMiscOff);  // abort flag; the waits' limit; TMEM address
    AttnRange* range = reinterpret_cast<AttnRange*>(base + L::kMiscOff + 16);
    AttnBars<SRC, D> bars{base_s + L::kBarOff};
    if (tid == 0) {
        for (int s = 0; s < L::kSlots; ++s) {
            mbar_init(bars.full(s), L::kPools ? 2 : 1);  // each warp that widens it, or the producer's expect_tx
            mbar_init(bars.empty(s), 2);                 // tcgen05.commit after each half's last MMA of the slot
        }
        for (int s = 0; s < L::kRaws; ++s) {
            mbar_init(bars.raw_full(s), 1);
            mbar_init(bars.raw_empty(s), 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bars.s_full(t), 1);
            mbar_init(bars.p_first(t), 4);
            mbar_init(bars.p_second(t), 4);
            mbar_init(bars.o_final(t), 1);
        }
        mbar_init(bars.q_full(), L::kPools ? 4 : 1);
        mbar_init(bars.q_empty(), 2);
        for (int t = 0; t < 2; ++t) {
            mbar_init(bars.drain(t), 1);
            mbar_init(bars.turn(t), 1);
            mbar_init(bars.piece_full(t), 1);
            mbar_init(bars.piece_empty(t), L::kPools ? 15 : 11);  // softmax 8, MMA 2, keys and values 1, widening 4
        }
        mbar_init(bars.tail(), 1);
        mbar_init(bars.odd_ml(), 4);
        mbar_init(bars.odd_read(), 4);
        fence_barrier_init();
        misc[0] = 0, misc[1] = p.wait_limit_ns;
    }
    if (warp == kAtMmaWarp) tmem_alloc(base_s + L::kMiscOff + 8, kAtTmemCols);
    pdl_wait_prerequisites();
    if constexpr (L::kPools) {
        if (tid == 0) p.cuts[blockIdx.x].w = -1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(base + L::kMiscOff + 8);
    if (L::kPools && warp >= kAtWidenWarp) {
        if constexpr (L::kPools) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kWidenRegs) : "memory");
            at_widen<SRC, D>(p, base, base_s, bars, misc, warp - kAtWidenWarp, lane);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoadRegs) : "memory");
        if (warp == kAtMmaWarp || warp == kAtMmaWarp + 1) {
            at_mma<SRC, D>(p, warp - kAtMmaWarp, base, base_s, tmem, bars, misc, lane);
        } else if constexpr (L::kPools) {
            if (warp == kAtKvWarp)
                at_load_raw<SRC, D>(p, base, base_s, bars, misc, lane);
            else
                at_walk<SRC, D>(p, range, base, bars, misc, lane);
        } else {
            if (warp == kAtKvWarp)
                at_load_packed<D>(p, &tmap_k, &tmap_v, base, base_s, bars, misc, lane);
            else
                at_load_q_packed<D>(p, &tmap_q, base, base_s, bars, misc, lane);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftmaxRegs) : "memory");
        at_softmax<SRC, D>(p, warp >> 2, base, tmem, bars, misc, warp, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kAtMmaWarp) tmem_dealloc(tmem, kAtTmemCols);
}

// Pools: the pieces of the unit that begins in CTA a = blockIdx.x and ends in CTA b, joined into out:
//     out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c,   M = max_c m_c,  in the CTAs' order.
// A warp takes kJoinRows rows, a lane per piece for the factors, then a lane per D / 32 elements; the factors' and the first
// pieces' loads are under way at once, for trips to L2 are what it costs.  A kernel of its own, on all SMs at once: the last
// CTA of a unit to end took 19 us for a join of 256 rows (4 sequences' turns over 32 KV heads, FP8: 179 us in all, 163 with
// this kernel; a mixed batch over 4-bit pools 33 and 23).  It is not let in before attn_kernel has ended: its blocks would
// wait beside the last CTAs (166).
constexpr int kJoinRows = 2, kJoinAhead = 4, kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 3) attn_join_kernel(const AttnParams p) {
    constexpr int E = D / 32;
    struct alignas(4 * E) Part {
        float x[E];
    };
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int4 cut = __ldcg(p.cuts + blockIdx.x);
    const int a = blockIdx.x, b = cut.w, lane = threadIdx.x & 31, rows = cut.y * p.group, tile_rows = p.tile_tokens * p.group;
    const int r0 = (blockIdx.y * kJoinWarps + threadIdx.x / 32) * kJoinRows;
    if (b < 0 || r0 >= rows) return;
    int64_t at[kJoinRows];  // the row's place in a slot's tiles
#pragma unroll
    for (int u = 0; u < kJoinRows; ++u) {
        const int r = min(r0 + u, rows - 1);
        at[u] = r >= tile_rows ? kAtRows + r - tile_rows : r;
    }
    auto slot = [&](int c) { return (int64_t)(2 * c + (c == a ? 1 : 0)) * p.part_tiles * kAtRows; };  // (a holds the unit's beginning)
    float m_at[kJoinRows];
    Part o[kJoinRows][kJoinAhead];
    // (a piece that sees none of a row's keys has stored no O: its factor is 0 and what is read there unused)
    auto fetch = [&](int c0) {
        const int mine = min(c0 + (lane & (kJoinAhead - 1)), b);
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) {
            m_at[u] = __ldcg(p.part_ml + slot(mine) + at[u]).x;
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                if (c0 + i > b) continue;
                const float* src = p.part_o + (slot(c0 + i) + at[u]) * D + lane * E;
                if constexpr (E == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
                    o[u][i] = Part{v.x, v.y, v.z, v.w};
                } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
                    o[u][i] = Part{v.x, v.y};
                }
            }
        }
    };
    float2 ml[kJoinRows];
    auto fetch_ml = [&](int c) {
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) ml[u] = __ldcg(p.part_ml + slot(min(c, b)) + at[u]);
    };
    fetch_ml(a + lane);
    fetch(a);
    float M[kJoinRows], L[kJoinRows], acc[kJoinRows][E];
#pragma unroll
    for (int u = 0; u < kJoinRows; ++u) M[u] = -INFINITY, L[u] = 0.f;
#pragma unroll 1
    for (int c = a + lane;; c += 32) {
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) {
            if (c > b) ml[u].x = -INFINITY;
            const float m = fmaxf(M[u], ml[u].x);
            if (m > -INFINITY) L[u] = L[u] * at_ref_exp2(M[u] - m) + ml[u].y * at_ref_exp2(ml[u].x - m);
            M[u] = m;
        }
        if (c - lane + 32 > b) break;
        fetch_ml(c + 32);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1)
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) {
            const float m2 = __shfl_xor_sync(0xffffffffu, M[u], x), l2 = __shfl_xor_sync(0xffffffffu, L[u], x);
            const float m = fmaxf(M[u], m2);
            if (m > -INFINITY) L[u] = L[u] * at_ref_exp2(M[u] - m) + l2 * at_ref_exp2(m2 - m);
            M[u] = m;
        }
#pragma unroll
    for (int u = 0; u < kJoinRows; ++u) {
        L[u] = p.out_scale / L[u];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[u][e] = 0.f;
    }
#pragma unroll 1
    for (int c0 = a;;) {
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) {
            const float f = m_at[u] > -INFINITY && c0 + (lane & (kJoinAhead - 1)) <= b ? at_ref_exp2(m_at[u] - M[u]) * L[u] : 0.f;
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                const float g = __shfl_sync(0xffffffffu, f, i);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[u][e] = g != 0.f ? acc[u][e] + g * o[u][i].x[e] : acc[u][e];
            }
        }
        c0 += kJoinAhead;
        if (c0 > b) break;
        fetch(c0);
    }
#pragma unroll
    for (int u = 0; u < kJoinRows; ++u) {
        const int r = r0 + u;
        if (r < rows) {
            const int tok = at_token(p, r);
            uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                        (((int64_t)cut.x + tok) * p.num_q_heads + (int64_t)cut.z * p.group + (r - tok * p.group)) * D + lane * E);
            if constexpr (E == 4)
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[u][0], acc[u][1]), pack_bf16x2(acc[u][2], acc[u][3]));
            else
                *dst = pack_bf16x2(acc[u][0], acc[u][1]);
        }
    }
}

bool aligned_to(const void* ptr, unsigned bytes) { return (reinterpret_cast<uintptr_t>(ptr) & (bytes - 1)) == 0; }

// One CTA per SM.
template <int SRC, int D>
pa_status launch_attn(const AttnParams& p, int dev, int grid, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                      cudaStream_t st) {
    using L = AttnLayout<SRC, D>;
    int occ = 0;
    if (!kernel_occupancy(dev, reinterpret_cast<const void*>(&attn_kernel<SRC, D>), L::kThreads, L::kBytes, &occ)) return PA_ERR_CUDA;
    if (occ <= 0) return PA_ERR_UNSUPPORTED;
    // The shares draw on what the launch gives, and with less the last one would be waited for for ever.  ptxas gives a kernel with
    // shares all that its launch bounds allow; a build where it did not is refused here.  (Shares that fit are enough.)
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes a;
        if (cudaFuncGetAttributes(&a, reinterpret_cast<const void*>(&attn_kernel<SRC, D>)) != cudaSuccess) return PA_ERR_CUDA;
        regs.store(a.numRegs);
    }
    if (regs.load() * (L::kThreads / 128) < 2 * L::kSoftmaxRegs + L::kLoadRegs + L::kWidenRegs) return PA_ERR_INTERNAL;
    if (launch_dependent(&attn_kernel<SRC, D>, dim3(grid), L::kThreads, L::kBytes, st, p, tq, tk, tv) != cudaSuccess) return PA_ERR_CUDA;
    if constexpr (L::kPools) {
        const dim3 join(grid, p.part_tiles * kAtRows / (kJoinRows * kJoinWarps));
        if (launch_dependent(&attn_join_kernel<D>, join, 32 * kJoinWarps, 0, st, p) != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

}  // namespace
}  // namespace pa
