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
    lib.t_most_packed_units.restype = ctypes.c_longlong
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
