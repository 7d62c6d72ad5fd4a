// How the chunk attention over quantised pools divides its work (host and device: plain integer arithmetic).
//
// A unit is two 128-row query tiles of one (sequence, KV head), or one; its work is the keys that its last row sees.
// Units are numbered sequence by sequence, KV head by KV head, from the first tokens to the last, and laid end to end on a
// line: a unit of `keys` keys takes U + keys * kTwoTiles of it, or U / 2 + keys * kOneTile, which adds up in closed form.
// U, a piece's fixed work, is the same for a whole call (unit_weight).
// CTA c of C takes the stages of 128 keys that begin in [c W / C, (c + 1) W / C).  Stage 0 begins with its unit, stage s > 0
// behind the unit's fixed part.  A range is never shorter than U + 2 * 128 (U / 2 + 128 in a call without units of two tiles),
// which is the longest distance of two stages' beginnings, so every CTA between the first and the last of a unit has a piece
// of it.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kAttnKeys = 128;   // keys per stage
constexpr int kAttnMaxLen = INT32_MAX - 255;  // longest sequence: a stage's keys, or two tiles' tokens, beyond it are still an int

// How many new tokens a sequence has whose rows are c0 .. end - 1 and which is len tokens long; none (and wrong) where it
// breaks the call's bounds.  The offsets may be anything, so that their difference may leave 32 bits: it is taken modulo 2^32
// and counts only where 0 <= c0 < end.  (INT32_MAX for len: its new tokens are all there is.)
PA_HD int sequence_tokens(int c0, int end, int len, int num_tokens, int max_new, int max_len, bool& wrong) {
    const int n = (int)((uint32_t)end - (uint32_t)c0);
    wrong = end < c0 || (end > c0 && (c0 < 0 || end > num_tokens || n > max_new || n > len || len > max_len));
    return wrong ? 0 : n;
}

// The most units of up to two tiles of T tokens that packed sequences can have, whatever their lengths within max_len and
// num_tokens in all: each one's full units, and one more where it has tokens.  (max_len alone, however loose, is no measure.)
PA_HD int64_t most_packed_units(int64_t num_seqs, int64_t num_tokens, int64_t max_len, int64_t kv_heads, int T) {
    const int64_t by_length = (max_len + 2 * T - 1) / (2 * T) * num_seqs;
    const int64_t by_tokens = num_tokens / (2 * T) + (num_seqs < num_tokens ? num_seqs : num_tokens);
    return (by_length < by_tokens ? by_length : by_tokens) * kv_heads;
}

constexpr int kTwoTiles = 2;     // weight of a key that two query tiles share
constexpr int kOneTile = 1;      // of one that a single tile uses
// U: a piece's query rows and epilogue take about as long as eight stages of one tile (4 sequences of 129 to 517 tokens over
// 32 KV heads of 128, FP8: 157 us with 1024, 163 with 512; 32 of 5 tokens over 8 heads: 111 and 114).  But the shortest range
// grows with U, so in a call of little work it is well below the largest with which every CTA still has a range (one short
// chunk: 22 us with 64, 17 with 2, which it gets; a mixed batch over 4-bit pools: 25 with that largest, 23 with an eighth of
// it), unless the units are so short that more of U makes more ranges (20 sequences of one token and up to 25 keys over 4
// heads: 63 us with 2, 17 with 1024).
constexpr int kUnitWeight = 1024;
// units: 1 for each of one tile, 2 for each of two
PA_HD int unit_weight(int64_t keys_weight, int64_t units, int64_t grid, bool one_tile) {
    if (keys_weight <= kAttnKeys * units) return kUnitWeight;
    // (keys_weight + units U / 2) / (U / 2 + 128 or twice that) >= grid
    const int64_t per = one_tile ? kOneTile : kTwoTiles, spare = keys_weight - per * kAttnKeys * grid, each = per * grid - units;
    if (each <= 0 || spare >= each * (kUnitWeight / 2)) return kUnitWeight;
    return spare < 8 * each ? 2 : 2 * (int)(spare / (8 * each));
}

// The units of one (sequence, KV head): n new tokens at the end of len, T tokens per tile.
struct UnitLine {
    int n, len, T, U;
    PA_HD int units() const { return (n + 2 * T - 1) / (2 * T); }
    PA_HD int two(int m) const { return 2 * m * T + T < n; }  // the unit's second tile has tokens
    PA_HD int keys(int m) const { return len - n + (2 * T * (m + 1) < n ? 2 * T * (m + 1) : n); }
    PA_HD int key_weight(int m) const { return two(m) ? kTwoTiles : kOneTile; }
    PA_HD int64_t weight(int m) const { return (two(m) ? U : U / 2) + (int64_t)keys(m) * key_weight(m); }
    // weight of the units before m (m < units(): all but the last unit have two tiles, and all their tokens)
    PA_HD int64_t before(int m) const {
        return (int64_t)m * (U + kTwoTiles * ((int64_t)(len - n) + (int64_t)T * (m + 1)));
    }
    PA_HD int64_t total() const {
        const int last = units() - 1;
        return last < 0 ? 0 : before(last) + weight(last);
    }
    // the last unit that begins at or before r
    PA_HD int unit_at(int64_t r) const {
        int lo = 0, hi = units() - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (before(mid) <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo;
    }
};

// The first stage that begins at or behind r of its unit.
PA_HD int64_t stage_at(int64_t r, int key_weight, int U) {
    if (r <= 0) return 0;
    if (key_weight == kOneTile) U /= 2;
    if (r <= U + key_weight * kAttnKeys) return 1;
    const int64_t k = r - U + key_weight * kAttnKeys - 1;
    return (key_weight == kTwoTiles ? k / kTwoTiles : k / kOneTile) / kAttnKeys;
}
PA_HD int64_t stage_begin(int64_t s, int key_weight, int U) { return s == 0 ? 0 : (key_weight == kOneTile ? U / 2 : U) + s * key_weight * kAttnKeys; }

PA_HD int64_t range_begin(int64_t c, int64_t W, int64_t C) { return c * W / C; }
PA_HD int64_t range_of(int64_t at, int64_t W, int64_t C) { return ((at + 1) * C - 1) / W; }
PA_HD int64_t ranges(int64_t W, int64_t grid, int U, bool one_tile) {
    const int64_t most = W / (one_tile ? U / 2 + kOneTile * kAttnKeys : U + kTwoTiles * kAttnKeys);
    return most < 1 ? 1 : most < grid ? most : grid;
}

}  // namespace pa
