"""CPU: the integer arithmetic of the prompt and chunk attention (csrc/pa_attn_plan.h, host and device code), compiled here and
compared with plain Python integers."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_280_gb300", "csrc")
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1

SHIM = r"""
#include "pa_attn_plan.h"
using namespace pa;
extern "C" {
int t_sequence(int c0, int end, int len, int num_tokens, int max_new, int max_len, int* wrong) {
    bool w;
    const int n = sequence_tokens(c0, end, len, num_tokens, max_new, max_len, w);
    *wrong = w;
    return n;
}
// The line of work of one call, then what every CTA of `grid` takes of it, walked as the kernel's roles walk it.  Units as
// (b, g, m, stages, key weight, beginning); pieces as (CTA, b, g, m, first stage, stages, cut_end or -1).  Returns the pieces' number,
// -1 if there are more than `room`.
long long t_unit_weight(const int* n, const int* len, int B, int H, int T, int grid, int one, long long* keys, long long* units) {
    long long W = 0, W2 = 0;
    for (int b = 0; b < B; ++b) W += UnitLine{n[b], len[b], T, 0}.total() * H, W2 += UnitLine{n[b], len[b], T, 2}.total() * H;
    *keys = W, *units = W2 - W;
    return unit_weight(W, W2 - W, grid, one);
}
void t_unit(int n, int len, int T, int U, int m, long long* out) {
    const UnitLine u{n, len, T, U};
    out[0] = u.units(), out[1] = u.total();
    if (m < u.units()) out[2] = u.keys(m), out[3] = u.key_weight(m), out[4] = u.weight(m), out[5] = u.before(m);
}
int t_unit_at(int n, int len, int T, int U, long long r) { return UnitLine{n, len, T, U}.unit_at(r); }
long long t_stage_at(long long r, int kw, int U) { return stage_at(r, kw, U); }
long long t_stage_begin(long long s, int kw, int U) { return stage_begin(s, kw, U); }
long long t_ranges(long long W, long long grid, int U, int one) { return ranges(W, grid, U, one); }
long long t_range_begin(long long c, long long W, long long C) { return range_begin(c, W, C); }
long long t_range_of(long long at, long long W, long long C) { return range_of(at, W, C); }
int t_pieces(const int* n, const int* len, int B, int H, int T, int U, long long W, long long C, int* out, int room) {
    int count = 0;
    for (long long c = 0; c < C; ++c) {
        const long long x = range_begin(c, W, C), end = range_begin(c + 1, W, C);
        long long before = 0;
        int b = 0;
        for (;; ++b) {  // the sequence in which the range begins, the KV head and the unit
            const long long w = UnitLine{n[b], len[b], T, U}.total() * H;
            if (x < before + w) break;
            before += w;
        }
        UnitLine u{n[b], len[b], T, U};
        int g = (int)((x - before) / u.total());
        long long r = (x - before) % u.total();
        int m = u.unit_at(r);
        r -= u.before(m);
        long long k = stage_at(r, u.key_weight(m), U), at = x - r;
        while (at < end) {
            u = UnitLine{n[b], len[b], T, U};
            if (u.units() == 0) {
                ++b;
                continue;
            }
            const long long stages = (u.keys(m) + kAttnKeys - 1) / kAttnKeys;
            const int kw = u.key_weight(m);
            const long long k0 = k < stages ? k : stages, reach = stage_at(end - at, kw, U), k1 = reach < stages ? reach : stages;
            if (k0 < k1) {
                if (count == room) return -1;
                int* p = out + 7 * count++;
                p[0] = (int)c, p[1] = b, p[2] = g, p[3] = m, p[4] = (int)k0, p[5] = (int)(k1 - k0);
                p[6] = k0 == 0 && k1 < stages ? (int)range_of(at + stage_begin(stages - 1, kw, U), W, C) : -1;
            }
            if (k1 < stages) break;
            at += u.weight(m), k = 0;
            if (++m == u.units()) {
                m = 0;
                if (++g == H) g = 0, ++b;
            }
        }
    }
    return count;
}
long long t_most_packed_units(int seqs, int tokens, int max_len, int kv_heads, int T) {
    return most_packed_units(seqs, tokens, max_len, kv_heads, T);
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    # signed overflow ends the process instead of wrapping unseen
    subprocess.check_call([cxx, "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)])
    lib = ctypes.CDLL(str(lib))
    for f in ("t_most_packed_units", "t_unit_weight", "t_stage_at", "t_stage_begin", "t_ranges", "t_range_begin", "t_range_of"):
        getattr(lib, f).restype = ctypes.c_longlong
    return lib


def test_tokens_of_sequences_whatever_the_offsets(plan):
    """Offsets and lengths around every bound and around the ends of 32 bits, differences past 32 bits among them."""
    wrong = ctypes.c_int()
    rng = random.Random(1)
    edges = [INT_MIN, INT_MIN + 1, INT_MIN + 5, -1000, -5, -1, 0, 1, 9, 10, 11, 99, 100, 101, 1 << 30, INT_MAX - 1, INT_MAX]
    calls = [(a, b, n, 100, 40, m) for a in edges for b in edges for n in (-7, 0, 5, 40, 41, 200, INT_MAX) for m in (40, INT_MAX)]
    calls += [tuple(rng.choice(edges) + rng.randint(0, 3) if rng.random() < 0.5 else rng.randint(0, 120) for _ in range(6))
              for _ in range(5000)]
    for call in calls:
        c0, end, length, tokens, new, longest = (max(INT_MIN, min(INT_MAX, x)) for x in call)
        n = end - c0
        bad = n < 0 or (n > 0 and (c0 < 0 or end > tokens or n > new or n > length or length > longest))
        got = plan.t_sequence(c0, end, length, tokens, new, longest, ctypes.byref(wrong))
        assert (got, bool(wrong.value)) == (0 if bad else n, bad), (c0, end, length, tokens, new, longest)


def test_most_units_of_packed_sequences(plan):
    """Never below the units that there are, and no more than their tokens allow where the bound on the lengths is loose."""
    rng = random.Random(2)
    for _ in range(3000):
        T, heads = 128 // rng.randint(1, 8), rng.randint(1, 70)
        top = rng.choice([1, 3, 40, 300, 5000])
        lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(rng.randint(1, 60))]
        tokens = sum(lens) + rng.randint(0, 9)
        loose = rng.choice([max(lens), tokens, max(lens) + rng.randint(0, 100)])
        there = sum(-(-n // (2 * T)) for n in lens) * heads
        most = plan.t_most_packed_units(len(lens), tokens, loose, heads, T)
        assert there <= most <= (tokens // (2 * T) + len(lens)) * heads
    assert plan.t_most_packed_units(65535, 66000, 66000, 8, 16) == 8 * (66000 // 32 + 65535)
    assert plan.t_most_packed_units(65535, INT_MAX, INT_MAX, 65535, 16) < 2 ** 43
    assert plan.t_most_packed_units(7, 4096, 33, 3, 16) == 7 * 2 * 3


def _i64(x):
    return ctypes.c_longlong(x)


def _ints(xs):
    return (ctypes.c_int * len(xs))(*xs)


def _unit(plan, n, length, T, U, m):
    out = (ctypes.c_longlong * 6)()
    plan.t_unit(n, length, T, U, m, out)
    return list(out)


def _units(n, length, T, U):
    """(keys, key weight, weight) of every unit of a sequence and KV head, by definition."""
    units = []
    for first in range(0, n, 2 * T):
        two = first + T < n  # the second tile has tokens
        keys = length - n + min(n, first + 2 * T)
        units.append((keys, 2 if two else 1, (U if two else U // 2) + keys * (2 if two else 1)))
    return units


def _batch(rng):
    T = 128 // rng.randint(1, 8)
    B, H, grid = rng.randint(1, 40), rng.randint(1, 6), rng.choice([1, 2, 7, 148, 152, rng.randint(1, 160)])
    top = rng.choice([1, 30, 130, 600, 5000, 40000])
    few = rng.choice([1, 1, 3, T, T + 1, 2 * T, 5 * T])
    lens = [rng.choice([1, 128, 129, top, rng.randint(1, top)]) for _ in range(B)]
    news = [0 if rng.random() < 0.2 else rng.randint(1, min(n, few)) for n in lens]
    one = max(news) <= T and rng.random() < 0.8  # what the host makes of its bound on the new tokens
    return T, H, grid, lens, news, one


def test_units_of_a_sequence(plan):
    rng = random.Random(3)
    for _ in range(400):
        T, _, _, lens, news, _ = _batch(rng)
        U = 2 * rng.randint(1, 512)
        for n, length in zip(news, lens):
            want = _units(n, length, T, U)
            at = 0
            for m, (keys, kw, weight) in enumerate(want):
                assert _unit(plan, n, length, T, U, m) == [len(want), sum(w[2] for w in want), keys, kw, weight, at]
                for r in {at, at + weight // 2, at + weight - 1}:
                    assert plan.t_unit_at(n, length, T, U, _i64(r)) == m
                at += weight
            if not want:
                assert _unit(plan, n, length, T, U, 0)[:2] == [0, 0]


def test_stages_begin_and_are_found(plan):
    rng = random.Random(4)
    for _ in range(3000):
        U, kw = 2 * rng.randint(1, 512), rng.choice([1, 2])
        s = rng.choice([0, 1, 2, rng.randint(0, 300), rng.randint(0, 2 ** 24)])
        begin = plan.t_stage_begin(_i64(s), kw, U)
        assert begin == (0 if s == 0 else U * kw // 2 + s * kw * 128)
        r = begin + rng.randint(-200, 200)
        got = plan.t_stage_at(_i64(r), kw, U)  # the first that begins at r or behind it
        assert got >= 0 and plan.t_stage_begin(_i64(got), kw, U) >= r
        assert got == 0 or plan.t_stage_begin(_i64(got - 1), kw, U) < r


@pytest.mark.parametrize("seed", range(6))
def test_every_stage_has_one_cta_and_every_piece_of_a_cut_unit_is_there(plan, seed):
    """Random batches: the pieces that the CTAs walk cover each stage of each unit once and in order; every CTA between the first
    and the last of a cut unit has a piece of it (the join reads one from each); the first names the last; a CTA begins one cut unit
    at most and continues one at most, its first piece; ranges are as long as two stages' beginnings may lie apart."""
    rng = random.Random(100 + seed)
    room = 200000
    out = (ctypes.c_int * (7 * room))()
    for _ in range(250):
        T, H, grid, lens, news, one = _batch(rng)
        n, length = _ints(news), _ints(lens)
        keys, units = ctypes.c_longlong(), ctypes.c_longlong()
        U = plan.t_unit_weight(n, length, len(news), H, T, grid, int(one), ctypes.byref(keys), ctypes.byref(units))
        want = [u for a, b in zip(news, lens) for u in _units(a, b, T, 0)]
        assert keys.value == H * sum(w for _, _, w in want) and units.value == H * sum(kw for _, kw, _ in want)
        assert 2 <= U <= 1024 and U % 2 == 0
        if rng.random() < 0.3:
            U = 2 * rng.randint(1, 512)  # the split holds for any
        W = H * sum(w for a, b in zip(news, lens) for _, _, w in _units(a, b, T, U))
        if W == 0:
            continue
        C = plan.t_ranges(_i64(W), _i64(grid), U, int(one))
        assert 1 <= C <= grid
        apart = U // 2 + 128 if one else U + 256
        begins = [plan.t_range_begin(_i64(c), _i64(W), _i64(C)) for c in range(C + 1)]
        assert begins[0] == 0 and begins[C] == W and (C == 1 or min(b - a for a, b in zip(begins, begins[1:])) >= apart)
        for c in range(C):
            for at in (begins[c], begins[c + 1] - 1):
                assert plan.t_range_of(_i64(at), _i64(W), _i64(C)) == c
        count = plan.t_pieces(n, length, len(news), H, T, U, _i64(W), _i64(C), out, room)
        assert count > 0
        pieces = [tuple(out[7 * i:7 * i + 7]) for i in range(count)]
        of_unit, of_cta = {}, {}
        for p in pieces:
            of_unit.setdefault(p[1:4], []).append(p)
            of_cta.setdefault(p[0], []).append(p)
        stages = {(b, g, m): -(-u[0] // 128) for b in range(len(news)) for m, u in enumerate(_units(news[b], lens[b], T, U))
                  for g in range(H)}
        assert set(of_unit) == set(stages)
        for unit, its in of_unit.items():
            assert [p[0] for p in its] == list(range(its[0][0], its[0][0] + len(its)))  # one CTA after another, none left out
            at = 0
            for p in its:
                assert p[4] == at and p[5] > 0
                at += p[5]
            assert at == stages[unit]
            assert [p[6] for p in its] == [its[-1][0] if len(its) > 1 else -1] + [-1] * (len(its) - 1)
        for c, its in of_cta.items():
            assert sum(p[6] >= 0 for p in its) <= 1 and all(p[4] == 0 for p in its[1:])
