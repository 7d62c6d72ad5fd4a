// How the chunk attention over quantised pools divides its work (host and device: plain integer arithmetic).
//
// A unit is two 128-row query tiles of one (sequence, KV head); its work is its stages of 128 keys.  Units are numbered
// sequence by sequence, KV head by KV head, from the first tokens to the last, and laid end to end on a line: a unit of
// nst stages takes kUnitWeight + nst * (kTwoTiles or kOneTile) of it.  CTA c of C takes the stages that begin in
// [c W / C, (c + 1) W / C).  Stage 0 begins with its unit, stage s > 0 behind the unit's fixed part.  A range is never
// shorter than kMinRange, which is more than the distance of two stages' beginnings, so every CTA between the first and
// the last of a unit has a piece of it.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kAttnKeys = 128;   // keys per stage
constexpr int kTwoTiles = 3;     // weight of a stage that two query tiles share
constexpr int kOneTile = 2;      // of one that a single tile uses
constexpr int kUnitWeight = 4;   // a piece's fixed work: query rows, epilogue
constexpr int kMinRange = 12;
static_assert(kMinRange >= kUnitWeight + kTwoTiles, "every CTA of a split unit has a piece");

// sum over i < n of floor((a i + b) / m), by exchanging the roles of the lattice's axes as in Euclid's algorithm.
PA_HD int64_t floor_sum(uint64_t n, uint64_t m, uint64_t a, uint64_t b) {
    uint64_t sum = 0;
    if (n == 0) return 0;
    for (;;) {
        if (a >= m) sum += n * (n - 1) / 2 * (a / m), a %= m;
        if (b >= m) sum += n * (b / m), b %= m;
        const uint64_t y = a * n + b;
        if (y < m) return (int64_t)sum;
        n = y / m, b = y % m;
        const uint64_t t = m;
        m = a, a = t;
    }
}

// The units of one (sequence, KV head): n new tokens at the end of len, T tokens per tile.
struct UnitLine {
    int n, len, T;
    PA_HD int units() const { return (n + 2 * T - 1) / (2 * T); }
    PA_HD int two(int m) const { return 2 * m * T + T < n; }  // the unit's second tile has tokens
    PA_HD int stages(int m) const {
        const int last = 2 * T * (m + 1) < n ? 2 * T * (m + 1) : n;
        return (int)(((int64_t)(len - n) + last + kAttnKeys - 1) / kAttnKeys);
    }
    PA_HD int stage_weight(int m) const { return two(m) ? kTwoTiles : kOneTile; }
    PA_HD int64_t weight(int m) const { return kUnitWeight + (int64_t)stages(m) * stage_weight(m); }
    // weight of the units before m (m < units(): all but the last unit have two tiles, and all their tokens)
    PA_HD int64_t before(int m) const {
        return (int64_t)m * kUnitWeight +
               kTwoTiles * floor_sum((uint64_t)m, kAttnKeys, 2u * T, (uint64_t)(len - n) + 2u * T + kAttnKeys - 1);
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
PA_HD int64_t stage_at(int64_t r, int stage_weight) {
    if (r <= 0) return 0;
    const int64_t s = (r - kUnitWeight + stage_weight - 1) / stage_weight;
    return s < 1 ? 1 : s;
}
PA_HD int64_t stage_begin(int64_t s, int stage_weight) { return s == 0 ? 0 : kUnitWeight + s * stage_weight; }

PA_HD int64_t range_begin(int64_t c, int64_t W, int64_t C) { return c * W / C; }
PA_HD int64_t range_of(int64_t at, int64_t W, int64_t C) { return ((at + 1) * C - 1) / W; }
PA_HD int64_t ranges(int64_t W, int64_t grid) {
    const int64_t most = W / kMinRange;
    return most < 1 ? 1 : most < grid ? most : grid;
}

}  // namespace pa
