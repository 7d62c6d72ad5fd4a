"""ORACLE -- test infrastructure only: the rotating append and the 4-bit pools, in numpy.

4-bit pool: bytes [num_blocks][Hkv][bs * (D / 2 + D / 16)]; a record holds the codes of its bs rows (element
2 j in the low half of byte j), then their E4M3 scale bytes.  value = E2M1(code) * E4M3(scale) * pool scale.
bf16 arrays are uint16 bit patterns, as elsewhere in the oracle.
"""
from __future__ import annotations

import numpy as np

import oracle

GROUP = 16
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def widen32(a: np.ndarray) -> np.ndarray:
    """bf16 bits or fp32 -> fp32 (exact)."""
    return (a.astype(np.uint32) << 16).view(np.float32) if a.dtype == np.uint16 else a.astype(np.float32)


def to_bf16(x: np.ndarray) -> np.ndarray:
    """fp32 -> bf16 bits, nearest even (NaN becomes a quiet NaN)."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    out = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), out)


def e2m1_value(codes: np.ndarray) -> np.ndarray:
    c = np.asarray(codes).astype(np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def e2m1_encode(x: np.ndarray) -> np.ndarray:
    """Nearest E2M1 code of each value; a tie takes the even code; saturates at 6; keeps the sign of zero."""
    a = np.abs(np.asarray(x, np.float64))[..., None]
    dist = np.abs(MAGNITUDES - np.minimum(a, 6.0))
    order = np.argsort(np.arange(8) % 2, kind="stable")  # even codes first
    best = order[np.argmin(dist[..., order], -1)]
    return (best + 8 * np.signbit(x)).astype(np.uint8)


def quantise_rows(x: np.ndarray, pool_scale: float):
    """fp32 rows [..][D] -> (code bytes [..][D / 2], scale bytes [..][D / 16])."""
    with np.errstate(all="ignore"):
        y = (np.asarray(x, np.float32) / np.float32(pool_scale)).reshape(*x.shape[:-1], -1, GROUP)
        nan = np.isnan(y).any(-1)
        amax = np.where(nan, np.float32(0), np.abs(np.where(np.isnan(y), 0, y)).max(-1)).astype(np.float32)
        sb = oracle.e4m3_encode(np.minimum(amax / np.float32(6), np.float32(448)))
        s = oracle.e4m3_value(sb).astype(np.float32)
        live = (s > 0) & ~nan
        z = y / np.where(live, s, np.float32(1))[..., None]
        codes = np.where(live[..., None], e2m1_encode(np.where(np.isnan(z), 0, z)), 0).astype(np.uint8)
    codes = codes.reshape(x.shape)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), np.where(nan, np.uint8(0x7F), sb)


def split(pool: np.ndarray, d: int, bs: int):
    """Views of a pool's code bytes [nb][Hkv][bs][D / 2] and scale bytes [nb][Hkv][bs][D / 16]."""
    nb, hkv, rec = pool.shape
    assert rec == bs * (d // 2 + d // GROUP)
    cut = bs * d // 2
    return pool[..., :cut].reshape(nb, hkv, bs, d // 2), pool[..., cut:].reshape(nb, hkv, bs, d // GROUP)


def append_fp4(k_new, v_new, k_pool, v_pool, slots, bs, k_scale, v_scale):
    """In-place append into 4-bit pools of the tokens whose slot is not negative."""
    d = k_new.shape[-1]
    cut = bs * d // 2
    for x, pool, scale in ((k_new, k_pool, k_scale), (v_new, v_pool, v_scale)):
        codes, scales = quantise_rows(widen32(x), scale)
        for i, s in enumerate(slots):
            if s >= 0:
                b, r = int(s) // bs, int(s) % bs
                pool[b, :, r * (d // 2): (r + 1) * (d // 2)] = codes[i]
                pool[b, :, cut + r * (d // GROUP): cut + (r + 1) * (d // GROUP)] = scales[i]


def values(pool: np.ndarray, d: int, bs: int) -> np.ndarray:
    """float64 [nb][Hkv][bs][D]: code * group scale, without the pool scale (exact)."""
    codes, scales = split(pool, d, bs)
    v = np.empty((*codes.shape[:-1], d))
    v[..., 0::2], v[..., 1::2] = e2m1_value(codes & 15), e2m1_value(codes >> 4)
    with np.errstate(invalid="ignore"):
        return v * np.repeat(oracle.e4m3_value(scales), GROUP, -1)


def decode_fp4(q, k_pool, v_pool, k_scale, v_scale, tables, lens, scale, bs, seqs=None):
    """float64 decode attention [B][Hq][D], and a bound on a kernel's error beside its output rounding.

    The bound is for weights rounded to f16 (relative 2^-11; 2^-36 of the largest below 2^-25 of it),
    fp32 dot products of D terms in any order (each term and partial sum off by 2^-22 of the terms'
    magnitudes: twice a rounding, for sums that a tensor core truncates), and 2^-18 for the exponentials
    and the merges' weights and sums.  With every weight off by a factor of at most 1 + e, the ratio of two
    sums of them is off by at most 2 e sum p |v|, to first order (e <= 1 / 64 here, so 2.1 covers it)."""
    B, hq, d = q.shape
    hkv = k_pool.shape[1]
    group = hq // hkv
    qf = widen32(q).astype(np.float64)
    out, bound = np.full((B, hq, d), np.nan), np.full((B, hq, d), np.nan)
    for b in range(B) if seqs is None else seqs:
        n = int(lens[b])
        out[b], bound[b] = 0.0, 0.0
        if n == 0:
            continue
        t = tables[b, : -(-n // bs)]
        k = values(k_pool[t], d, bs).transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] * np.float64(np.float32(k_scale))
        v = values(v_pool[t], d, bs).transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] * np.float64(np.float32(v_scale))
        for h in range(hq):
            kh, vh = k[h // group], v[h // group]
            x = kh @ qf[b, h] * scale
            p = np.exp(x - x.max())
            p /= p.sum()
            size = (np.abs(kh) @ np.abs(qf[b, h]) * abs(scale)).max()
            e = 2.0 ** -11 + d * 2.0 ** -22 * size + 2.0 ** -18
            out[b, h] = p @ vh
            # weights below 2^-25 of the largest one, which is held as 2^11 at least: an absolute 2^-36 of it each
            tiny = 2.0 ** -36 * p.max() * np.abs(vh).sum(0)
            bound[b, h] = 2.1 * e * (p @ np.abs(vh)) + 2 * tiny
    return out, bound


def rotate_exact(x, positions, cos_sin, interleaved):
    """x [N][H][D] turned, in float64."""
    return _rotate(widen32(x).astype(np.float64), positions, cos_sin.astype(np.float64), interleaved)


def rotate_f32(x, positions, cos_sin, interleaved):
    """x [N][H][D] turned, in fp32 with every product and sum rounded."""
    return _rotate(widen32(x), positions, cos_sin.astype(np.float32), interleaved)


def _rotate(x, positions, cos_sin, interleaved):
    half = cos_sin.shape[1] // 2
    y = x.copy()
    for i, p in enumerate(positions):
        for j in range(half):
            ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = cos_sin[p, j], cos_sin[p, half + j]
            a, b = x[i, :, ia], x[i, :, ib]
            y[i, :, ia] = a * c - b * s
            y[i, :, ib] = b * c + a * s
    return y


def cos_sin_table(max_position: int, rot_dim: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [max_position][rot_dim]: cos then sin of p * base^(-2 j / rot_dim), the angles in float64."""
    j = np.arange(rot_dim // 2)
    a = np.arange(max_position)[:, None] * base ** (-2.0 * j / rot_dim)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
