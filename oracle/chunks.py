"""ORACLE -- test infrastructure only: attention of several query rows per sequence, and the head norms, in numpy float64.

bf16 arrays are uint16 bit patterns, as elsewhere in the oracle.
"""
from __future__ import annotations

import numpy as np

import oracle
from oracle import kv4

EPS_BF16, EPS_F16 = 2.0 ** -8, 2.0 ** -11  # half a step, relative


def causal(q, k, v, first, scale, weight_eps):
    """One sequence: q [n][Hq][D], k / v [T][Hkv][D] float64, row i at position first + i -> (out [n][Hq][D], bound).

    The bound is on a kernel's error beside its output rounding.  The weights enter the product with V rounded (relative
    weight_eps; 2^-32 of the largest where f16 runs out of exponents), but not the sum that divides it.  Both hold
    exponentials of scores off by D terms of 2^-22 each of the magnitudes (fp32 sums that a tensor core truncates) and by
    what scaling the query row into f16 may drop (2^-25 of its largest element each), another 2^-18 for the exponential,
    the shared maximum and the joins, and fp32 sums over the keys (2^-24 a key).  A factor of at most 1 + e on every
    weight moves the ratio by at most 2 e sum p |v| to first order (2.1 covers e <= 1 / 64)."""
    n, hq, d = q.shape
    hkv = k.shape[1]
    out, bound = np.empty(q.shape), np.empty(q.shape)
    late = np.arange(len(k))[None] > first + np.arange(n)[:, None]
    for h in range(hq):
        kh, vh, qh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], q[:, h]
        x = np.where(late, -np.inf, qh @ kh.T * scale)
        p = np.exp(x - x.max(1, keepdims=True))
        top = 1 / p.sum(1, keepdims=True)
        p *= top
        seen_k = np.abs(kh)[: first + n]
        size = (np.abs(qh) @ seen_k.T * scale).max(1, keepdims=True)
        lost = 2.0 ** -25 * np.abs(qh).max(1, keepdims=True) * seen_k.sum(1).max() * scale
        e = d * 2.0 ** -22 * size + lost + 2.0 ** -18 + len(k) * 2.0 ** -24
        pv = p @ np.abs(vh)
        out[:, h] = p @ vh
        bound[:, h] = (weight_eps + 2.1 * e) * pv + 2.0 ** -32 * top * np.abs(vh).sum(0)
    return out, bound


def prompts(q, k, v, starts, scale):
    """Packed prompts: q [T][Hq][D], k / v [T][Hkv][D] bf16 bits -> (out, bound) float64, NaN in rows of no sequence."""
    out, bound = (np.full(q.shape, np.nan) for _ in range(2))
    for a, e in zip(starts[:-1], starts[1:]):
        if e > a:
            x = [kv4.widen32(t[a:e]).astype(np.float64) for t in (q, k, v)]
            out[a:e], bound[a:e] = causal(*x, 0, scale, EPS_BF16)
    return out, bound


def pool_values(pool, kind, d, bs):
    """float64 [nb][Hkv][bs][D] of a quantised pool, without the pool scale."""
    return oracle.e4m3_value(pool).astype(np.float64) if kind == "fp8" else kv4.values(pool, d, bs)


def chunks(q, k_pool, v_pool, kind, k_scale, v_scale, tables, lens, starts, scale, bs, seqs=None):
    """Chunk attention over a quantised pool: q [T][Hq][D] bf16 bits -> (out, bound) float64."""
    d = q.shape[2]
    out, bound = (np.full(q.shape, np.nan) for _ in range(2))
    for b in range(len(lens)) if seqs is None else seqs:
        a, e, t = int(starts[b]), int(starts[b + 1]), int(lens[b])
        if e <= a:
            continue
        table = tables[b, : -(-t // bs)]
        k, v = (pool_values(p[table], kind, d, bs).transpose(0, 2, 1, 3).reshape(-1, p.shape[1], d)[:t] * np.float64(np.float32(s))
                for p, s in ((k_pool, k_scale), (v_pool, v_scale)))
        out[a:e], bound[a:e] = causal(kv4.widen32(q[a:e]).astype(np.float64), k, v, t - (e - a), scale, EPS_F16)
    return out, bound


def head_norm(x, w, eps):
    """x [N][H][D] (bf16 bits or fp32) normed per head and weighted, in float64."""
    x = kv4.widen32(x).astype(np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
