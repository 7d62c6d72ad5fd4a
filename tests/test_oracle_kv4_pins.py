"""Pins of the oracle's 4-bit codes, group quantiser, unpacking and decode, and of its rotation."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4
import oracle


def _magnitude(code):
    """E2M1 from its bit layout: exponent bias 1, one mantissa bit."""
    e, m = code >> 1, code & 1
    return Fraction(m, 2) if e == 0 else (1 + Fraction(m, 2)) * 2 ** (e - 1)


def test_code_table():
    assert [Fraction(float(v)) for v in kv4.e2m1_value(np.arange(8))] == [_magnitude(c) for c in range(8)]
    assert np.array_equal(kv4.e2m1_value(np.arange(8, 16)), -kv4.e2m1_value(np.arange(8)))


def test_encoder_matches_exact_search():
    mags = [_magnitude(c) for c in range(8)]
    ties = [(a + b) / 2 for a, b in zip(mags, mags[1:])]
    rng = np.random.default_rng(0)
    xs = np.array([float(x) for x in mags + ties] + [5.001, 7.0, 1e30] + list(rng.uniform(0, 7, 400)), np.float32)
    xs = np.concatenate([xs, np.nextafter(xs, np.float32(0)), np.nextafter(xs, np.float32(10))])
    for x, got in zip(np.concatenate([xs, -xs]), kv4.e2m1_encode(np.concatenate([xs, -xs]))):
        a = min(abs(Fraction(float(x))), Fraction(6))
        want = min(range(8), key=lambda c: (abs(mags[c] - a), c & 1))
        assert got == want + (8 if np.signbit(x) else 0), x


def test_e4m3_encoder_saturates_at_any_size():
    x = np.array([448.0, 464.0, 1e4, 2.0 ** 62, 1e30, np.inf], np.float32)
    assert oracle.e4m3_encode(np.concatenate([x, -x])).tolist() == [0x7E] * 6 + [0xFE] * 6


@pytest.mark.parametrize("pool_scale", [1.0, 0.043, 3.7])
def test_group_quantiser(pool_scale):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)) * 2)).astype(np.float32)
    codes, scales = kv4.quantise_rows(x, pool_scale)
    rec = np.concatenate([codes.reshape(-1), scales.reshape(-1)])
    # as one record of 50 rows (the layout's block size is free in the oracle)
    v = kv4.values(rec[None, None], 128, 50)[0, 0] * np.float32(pool_scale)
    amax = np.abs(x).reshape(50, -1, 16).max(-1)
    step = np.repeat(oracle.e4m3_value(scales) * np.float32(pool_scale), 16, -1).reshape(50, 128)
    # The scale is within half a step (2^-4) of amax / 6, or 2^-10 absolute.  An element within 6 scales is at
    # most half the codes' widest gap off, one scale.  A larger one saturates: it is off by at most
    # amax - 6 s <= 6 |amax / 6 - s| <= amax 2^-4 + 6 * 2^-10, and amax < 2 |x| there unless the scale rounds
    # to zero, where amax itself is below 6 * 2^-10.
    assert np.all(np.abs(oracle.e4m3_value(scales) * pool_scale - amax / 6) <= amax / 6 * 2.0 ** -4 * 1.0001 + pool_scale * 2.0 ** -10)
    assert np.all(np.abs(v - x) <= step * 1.0001 + 2.0 ** -3 * np.abs(x) + pool_scale * 6 * 2.0 ** -10 * 1.0001)


def test_group_edge_values():
    x = np.zeros((5, 64), np.float32)
    x[1, 3] = np.nan
    x[2, 20] = np.inf
    x[3] = 1e-9       # the scale rounds to zero
    x[4, :16] = 2.0 ** -9 * 6 * np.linspace(-1, 1, 16)
    codes, scales = kv4.quantise_rows(x, 1.0)
    assert scales[0].tolist() == [0] * 4 and not codes[0].any() and not codes[3].any()
    assert scales[1, 0] == 0x7F and not codes[1].any() and scales[1, 1] == 0
    assert scales[2, 1] == 0x7E and codes[2, 10] == 7 and np.count_nonzero(codes[2]) == 1
    assert scales[4, 0] == 1 and codes[4, 0] & 15 == 15 and codes[4, 7] >> 4 == 7


def test_append_and_values_round_trip():
    rng = np.random.default_rng(2)
    for d, bs in ((64, 16), (128, 32)):
        kp = rng.integers(0, 256, (5, 2, bs * (d // 2 + d // 16))).astype(np.uint8)
        vp, before = kp.copy(), kp.copy()
        # rows of representable values come back exactly
        x = (kv4.e2m1_value(rng.integers(0, 16, (7, 2, d))) * 0.5).astype(np.float32)
        x[..., ::16] = 3.0  # each group's largest is 6 * 0.5
        slots = np.array([3, bs + 1, 2 * bs, -1, 4 * bs + bs - 1, 5, 9])
        kv4.append_fp4(x, -x, kp, vp, slots, bs, 0.25, 2.0)
        kv, vv = kv4.values(kp, d, bs) * 0.25, kv4.values(vp, d, bs) * 2.0
        for i, s in enumerate(slots):
            if s >= 0:
                assert np.array_equal(kv[s // bs, :, s % bs], x[i]) and np.array_equal(vv[s // bs, :, s % bs], -x[i])
        codes, scales = kv4.split(kp, d, bs)
        c0, s0 = kv4.split(before, d, bs)
        keep = np.ones((5, bs), bool)
        for s in slots[slots >= 0]:
            keep[s // bs, s % bs] = False
        assert np.array_equal(codes.transpose(0, 2, 1, 3)[keep], c0.transpose(0, 2, 1, 3)[keep])
        assert np.array_equal(scales.transpose(0, 2, 1, 3)[keep], s0.transpose(0, 2, 1, 3)[keep])


def test_decode_closed_forms():
    rng = np.random.default_rng(3)
    d, bs, hkv, hq = 64, 16, 2, 4
    kp = rng.integers(0, 256, (4, hkv, bs * 36)).astype(np.uint8)
    vp = rng.integers(0, 256, (4, hkv, bs * 36)).astype(np.uint8)
    for p in (kp, vp):
        p[..., bs * 32:] = rng.integers(0x20, 0x48, p[..., bs * 32:].shape)
    q = rng.standard_normal((3, hq, d)).astype(np.float32)
    tables = np.array([[2, 0], [1, 3], [0, 0]], np.int32)
    out, bound = kv4.decode_fp4(q, kp, vp, 0.5, 0.25, tables, np.array([1, 20, 0]), 0.1, bs)
    v = kv4.values(vp, d, bs) * 0.25
    assert np.array_equal(out[0], v[2, :, 0].repeat(2, 0)) and not out[2].any() and not bound[2].any()
    kp[1], kp[3] = 0, 0  # all keys zero: the mean of the values
    out, _ = kv4.decode_fp4(q, kp, vp, 0.5, 0.25, tables, np.array([1, 20, 0]), 0.1, bs)
    mean = np.concatenate([v[1], v[3][:, :4]], 1).mean(1)
    assert np.allclose(out[1], mean.repeat(2, 0), rtol=0, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    rng = np.random.default_rng(4)
    rot, d = 32, 64
    table = kv4.cos_sin_table(50, rot)
    x = rng.standard_normal((4, 3, d)).astype(np.float32)
    y = kv4.rotate_exact(x, [0, 1, 7, 49], table, interleaved)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., rot:], x[..., rot:])
    # each pair turns by its angle: a complex product
    pair = (lambda a: a[..., 0:rot:2] + 1j * a[..., 1:rot:2]) if interleaved else (lambda a: a[..., : rot // 2] + 1j * a[..., rot // 2: rot])
    ang = np.array([0, 1, 7, 49])[:, None] * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    assert np.allclose(pair(y), pair(x) * np.exp(1j * ang)[:, None], rtol=0, atol=2e-6)
    # the product of two turned rows depends on the distance of their positions only
    a = [kv4.rotate_exact(x[:1], [p], table, interleaved)[0, 0] @ kv4.rotate_exact(x[1:2], [p + 5], table, interleaved)[0, 0]
         for p in (0, 11, 44)]
    assert np.allclose(a, a[0], rtol=0, atol=1e-5)
    f = kv4.rotate_f32(x, [0, 1, 7, 49], table, interleaved)
    assert f.dtype == np.float32 and np.all(np.abs(f - y) <= 2.0 ** -23 * np.abs(x).max() * 3)
