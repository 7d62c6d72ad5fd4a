"""GPU: 4-bit decode where the softmax is at its extremes."""
import numpy as np
import pytest

from gpu_cases import status_word, to_numpy, to_torch, widen
from oracle import kv4

pytestmark = pytest.mark.gpu


def _decode(q, kp, vp, tables, lens, scale, ks=1.0, vs=1.0, part=0):
    import torch
    import paged_kv_cache_280_gb300 as pa

    b, hq, d = q.shape
    out = torch.full_like(q, float("nan"))
    ws = torch.zeros(pa.pa_decode_workspace_bytes(b, hq, kp.shape[1], d), dtype=torch.uint8, device="cuda")
    pa.pa_decode_attention_fp4(out, q, kp, vp, ks, vs, tables, lens, int(lens.max()), scale, ws, partition_tokens=part)
    assert status_word(ws) == 0
    return widen(to_numpy(out))


def _far_apart(size, d, bs, hkv):
    """Sequences whose keys are zero but for two random ones, and queries of the given size."""
    group = 8
    rng = np.random.default_rng(int(np.log2(size)) + d)
    lens = np.array([600, 1, 77, 600], np.int32)
    need = -(-lens // bs)
    tables = np.zeros((len(lens), need.max()), np.int32)
    kp = np.zeros((need.sum(), hkv, bs * (d // 2 + d // 16)), np.uint8)
    vp = rng.integers(0, 256, kp.shape).astype(np.uint8)
    cut = bs * d // 2
    vp[..., cut:] = rng.integers(0x20, 0x41, vp[..., cut:].shape)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = at + rng.permutation(n)
        at += n
        for t in {0, int(lens[b]) * 2 // 3}:  # (one key where a sequence has one token)
            block, r = kp[tables[b, t // bs]], t % bs
            block[:, r * (d // 2): (r + 1) * (d // 2)] = rng.integers(0, 256, (hkv, d // 2))
            block[:, cut + r * (d // 16): cut + (r + 1) * (d // 16)] = rng.integers(0x30, 0x41, (hkv, d // 16))
    q = kv4.to_bf16((rng.standard_normal((len(lens), group * hkv, d)) * size).astype(np.float32))
    return q, kp, vp, tables, lens


def _one_hot(q, kp, vp, tables, lens, scale, bs):
    """float64 outputs of a softmax that gives all weight to the largest score, and the mean |value| under it.  Asserts
    that the largest score is ahead of the rest: by 64, and by twice what fp32 dot products of d terms may be off (2^-22 of
    the terms' magnitudes each)."""
    hq, d = q.shape[1:]
    hkv = kp.shape[1]
    k, v = (kv4.values(p, d, bs) for p in (kp, vp))
    ref, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        t = tables[b, : -(-n // bs)]
        kb, vb = (p[t].transpose(1, 0, 2, 3).reshape(hkv, -1, d)[:, :n] for p in (k, v))
        for h in range(hq):
            kh, vh, qh = kb[h * hkv // hq], vb[h * hkv // hq], kv4.widen32(q[b, h]).astype(np.float64)
            x = kh @ qh * scale
            off = d * 2.0 ** -22 * (np.abs(kh) @ np.abs(qh) * abs(scale)).max()
            top = x == x.max()
            assert top.all() or x.max() - x[~top].max() > max(64.0, 2 * off)
            ref[b, h], mag[b, h] = vh[top].mean(0), np.abs(vh[top]).mean(0)
    return ref, mag


SIZES = [2.0 ** 22, 3e8, 1e10, 1e20, 1e34]


@pytest.mark.parametrize("part", [0, 64])
@pytest.mark.parametrize("size", [1.0] + SIZES)
@pytest.mark.parametrize("d,bs,hkv", [(128, 16, 1), (64, 32, 2)])
def test_scores_of_any_size(size, d, bs, hkv, part):
    """Scores of sizes at which fp32 no longer tells neighbouring whole numbers apart, under both signs of the score
    scale: the largest takes all the weight, shared by the keys of zero where it is theirs."""
    q, kp, vp, tables, lens = _far_apart(size, d, bs, hkv)
    for scale in (0.3, -0.3):
        got = _decode(*(to_torch(x) for x in (q, kp, vp, tables, lens)), scale, part=part)
        if size == 1.0:
            ref, loose = kv4.decode_fp4(q, kp, vp, 1.0, 1.0, tables, lens, scale, bs)
        else:  # equal weights, and sums of up to 600 terms in fp32 (2^-23 of the sum each, if a tensor core truncates)
            ref, mag = _one_hot(q, kp, vp, tables, lens, scale, bs)
            loose = 2 * 600 * 2.0 ** -23 * mag
        err = np.abs(got - ref)
        assert np.all(err <= 2.0 ** -8 * (np.abs(ref) + loose) + loose), (np.isnan(got).sum(), np.nanmax(err))


@pytest.mark.parametrize("part", [0, 256])
def test_the_pool_scale_of_the_values_is_of_any_size(part):
    """A power of two in the values' pool scale comes out in the outputs, down to where a bf16 output is still normal."""
    rng = np.random.default_rng(3)
    d, bs, hkv, lens = 128, 16, 2, np.array([40000, 3, 0, 900], np.int32)
    kp, vp = (rng.integers(0, 256, (50, hkv, bs * 72)).astype(np.uint8) for _ in range(2))
    for p in (kp, vp):
        p[..., bs * 64:] = rng.integers(0x28, 0x39, p[..., bs * 64:].shape)
    vp[..., : bs * 64] &= 0x77                 # positive values,
    vp[..., : bs * 64] |= 0x22                 # of at least 1
    vp[..., bs * 64:] += 0x30                  # times 16 and more
    tables = rng.integers(0, 50, (4, 2500)).astype(np.int32)
    q = kv4.to_bf16(rng.standard_normal((4, 8, d)).astype(np.float32))
    args = [to_torch(x) for x in (q, kp, vp, tables, lens)]
    one, small = (_decode(*args, 0.09, vs=s, part=part) for s in (1.0, 2.0 ** -125))
    assert one[lens > 0].min() > 1.0 and np.array_equal(small, one * 2.0 ** -125)


@pytest.mark.parametrize("n,drop", [(131072, 24.4), (131072, 25.01), (1 << 20, 25.01), (1 << 20, 33.0)])
def test_a_long_tail_of_small_weights(n, drop):
    """One key ahead of n - 1 equal ones by `drop` powers of two: their share, (n - 1) 2^-drop of the first's, is not lost.
    As many segments as there are warps, so that a warp takes a whole one; the tables repeat two blocks."""
    import torch

    d, bs, hkv = 64, 32, 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B = -(-sms * 16 * 5 // 4 // hkv)
    kp, vp = (np.zeros((2, hkv, bs * 36), np.uint8) for _ in range(2))
    codes = bs * d // 2
    kp[0, :, 0], kp[0, :, codes] = 0x02, 0x38                    # the first key: 1 in dim 0; all others 0
    vp[..., :codes], vp[..., codes:] = 0x22, 0x38                # every value 1 ..
    vp[0, :, : d // 2] = 0                                       # .. but the first, 0
    q = torch.zeros(B, hkv, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    tables = torch.ones(B, n // bs, dtype=torch.int32, device="cuda")
    tables[:, 0] = 0
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    got = _decode(q, to_torch(kp), to_torch(vp), tables, lens, drop * np.log(2.0))
    tail = (n - 1) * 2.0 ** -drop
    want = tail / (1.0 + tail)
    # the output's rounding; f16 weights, 2^-11 each or, below 2^-25 of the largest, 2^-36 of it (twice, for two sums);
    # and the two sums in fp32 by the tensor cores, which align a step's products with the sum they join and cut each
    # of them there: n terms, each off by up to 2^-23 of the sum
    lim = (2.0 ** -8 + 2 * (2.0 ** -11 + n * 2.0 ** -23)) * want + 2 * n * 2.0 ** -36
    assert np.abs(got - want).max() <= lim, f"{np.abs(got - want).max():.3e} off at {want:.3e}, {lim:.3e} allowed"
