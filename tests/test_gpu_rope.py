"""GPU: the rotating append (pa_rope_and_cache) into every pool type, bit-exact against the oracle's fp32 rotation
and quantisers, and within one rounding of the rotation in float64."""
import numpy as np
import pytest

import oracle
import synth
from gpu_cases import to_numpy, to_torch, widen
from oracle import kv4

pytestmark = pytest.mark.gpu

MAXP = 300


def _inputs(seed, n, hq, hkv, d, dtype, fused):
    h = hq + 2 * hkv
    x = synth.normal(synth.stream_seed(seed, 1), n * h * d, dtype).reshape(n, h, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if fused:
        t = to_torch(x)
        dev = (t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:])
    else:
        dev = tuple(to_torch(np.ascontiguousarray(a)) for a in (q, k, v))
    return (q, k, v), dev


def _pool(seed, nb, hkv, bs, d, pool):
    if pool == "fp4":
        return np.random.default_rng(seed).integers(0, 256, (nb, hkv, bs * (d // 2 + d // 16))).astype(np.uint8)
    if pool == "fp8":
        return np.random.default_rng(seed).integers(0, 256, (nb, hkv, bs, d)).astype(np.uint8)
    return synth.normal(synth.stream_seed(seed, 9), nb * hkv * bs * d, pool).reshape(nb, hkv, bs, d)


def _round(x, dtype):
    return x if dtype == "f32" else kv4.to_bf16(x)


def _oracle_append(pool, kp, vp, k, v, slots, bs, ks, vs):
    """k (fp32, turned) and v (fp32) into host pools."""
    kept = slots >= 0
    if pool == "fp4":
        kv4.append_fp4(k[kept], v[kept], kp, vp, slots[kept], bs, ks, vs)
    elif pool == "fp8":
        oracle.reshape_and_cache_fp8(k[kept], v[kept], kp, vp, slots[kept], ks, vs)
    else:
        oracle.reshape_and_cache(_round(k[kept], pool), _round(v[kept], pool), kp, vp, slots[kept])


CASES = [
    # n, hq, hkv, d, bs, in, pool, rot, interleaved, fused
    (1, 8, 2, 128, 16, "bf16", "bf16", 128, False, True),
    (1, 1, 1, 64, 32, "f32", "f32", 64, True, False),
    (37, 32, 8, 128, 16, "bf16", "bf16", 128, False, True),
    (37, 5, 5, 64, 32, "bf16", "bf16", 32, False, False),
    (37, 6, 3, 128, 32, "bf16", "bf16", 48, False, True),   # an odd number of rotating units per row
    (29, 6, 2, 128, 16, "bf16", "bf16", 64, True, True),
    (23, 4, 4, 64, 16, "f32", "f32", 64, False, False),
    (23, 7, 1, 128, 16, "f32", "f32", 16, True, True),
    (31, 8, 8, 128, 16, "bf16", "fp8", 128, False, True),
    (31, 16, 2, 128, 32, "f32", "fp8", 64, True, False),
    (33, 8, 2, 128, 16, "bf16", "fp4", 128, False, True),
    (33, 3, 3, 64, 32, "bf16", "fp4", 32, False, True),
    (33, 4, 2, 64, 16, "f32", "fp4", 64, True, False),
    (33, 12, 4, 128, 32, "f32", "fp4", 96, False, True),
    (700, 32, 8, 128, 16, "bf16", "fp4", 128, False, True),  # more rows than one turn of the grid
]


@pytest.mark.parametrize("n,hq,hkv,d,bs,dtype,pool,rot,inter,fused", CASES)
def test_rope_append_bit_exact(n, hq, hkv, d, bs, dtype, pool, rot, inter, fused):
    import torch
    import paged_kv_cache_280_gb300 as pa

    seed = 1000 + n + hq + d + rot
    (q, k, v), (dq, dk, dv) = _inputs(seed, n, hq, hkv, d, dtype, fused)
    nb = -(-n // bs) + 3
    slots = synth.permutation(seed, nb * bs)[:n].astype(np.int64)
    if n > 5:
        slots[[2, n - 1]] = -1  # padding
    pos = synth.uniform_ints(seed + 1, n, 0, MAXP - 1).astype(np.int32)
    pos[0] = MAXP - 1
    if n > 5:
        pos[2] = -5  # a padding token's position is not looked at
    table = kv4.cos_sin_table(MAXP, rot)
    kp, vp = _pool(seed, nb, hkv, bs, d, pool), _pool(seed + 7, nb, hkv, bs, d, pool)
    dkp, dvp = to_torch(kp), to_torch(vp)
    ks, vs = 0.037, 1.75
    q_out = to_torch(_pool(3, n, hq, 1, d, dtype).reshape(n, hq, d))
    q_before = to_numpy(q_out).copy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_and_cache(q_out, dq, dk, dv, to_torch(pos), to_torch(table), dkp, dvp, to_torch(slots), interleaved=inter,
                         k_scale=ks, v_scale=vs, status=status)
    safe = np.where(slots >= 0, pos, 0)
    rq, rk = kv4.rotate_f32(q, safe, table, inter), kv4.rotate_f32(k, safe, table, inter)
    want_q = np.where((slots >= 0)[:, None, None], _round(rq, dtype), q_before)
    _oracle_append(pool, kp, vp, rk, kv4.widen32(v), slots, bs, ks, vs)
    assert status.item() == 0
    assert np.array_equal(to_numpy(q_out), want_q)
    assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
    # and against float64: two products and a sum in fp32 (2^-24 each of |a c| + |b s| <= 2 max|x|), then one rounding
    exact = kv4.rotate_exact(q, safe, table, inter)
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    err = np.abs(widen(to_numpy(q_out)) - exact)[slots >= 0]
    size = np.abs(kv4.widen32(q)).max()
    assert np.all(err <= half * np.abs(exact[slots >= 0]) + 3 * 2.0 ** -24 * 2 * size * (1 + half))


def test_rope_in_place_and_without_queries():
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 19, 8, 2, 128, 16, 4
    (q, k, v), (dq, dk, dv) = _inputs(5, n, hq, hkv, d, "bf16", False)
    slots = np.arange(n, dtype=np.int64) + 3
    pos = np.arange(n, dtype=np.int32)
    table = to_torch(kv4.cos_sin_table(MAXP, d))
    pools = [torch.zeros(nb, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    apart = torch.empty_like(dq)
    pa.pa_rope_and_cache(apart, dq, dk, dv, to_torch(pos), table, pools[0], pools[1], to_torch(slots))
    pa.pa_rope_and_cache(None, None, dk, dv, to_torch(pos), table, pools[2], pools[3], to_torch(slots))
    pa.pa_rope_and_cache(dq, dq, dk, dv, to_torch(pos), table, pools[0], pools[1], to_torch(slots))
    assert torch.equal(dq, apart) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert np.array_equal(to_numpy(apart), kv4.to_bf16(kv4.rotate_f32(q, pos, kv4.cos_sin_table(MAXP, d), False)))


@pytest.mark.parametrize("pool", ["bf16", "fp4"])
def test_rope_flags_bad_slots_and_positions(pool):
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 5, 4, 2, 64, 16, 3
    (q, k, v), (dq, dk, dv) = _inputs(6, n, hq, hkv, d, "bf16", True)
    table = kv4.cos_sin_table(MAXP, d)
    for slots, pos, flag in (([1, nb * bs, 3, 4, 5], [1, 2, 3, 4, 5], pa.PA_DEV_BAD_SLOT),
                             ([1, 2, 3, 4, 5], [1, MAXP, 3, 4, 5], pa.PA_DEV_BAD_POSITION),
                             ([1, 2, 3, 4, 5], [1, -1, 3, 4, 5], pa.PA_DEV_BAD_POSITION),
                             ([1, 1 << 40, 3, 4, 5], [1, -1, 3, 4, 5], pa.PA_DEV_BAD_SLOT | pa.PA_DEV_BAD_POSITION)):
        kp, vp = _pool(1, nb, hkv, bs, d, pool), _pool(2, nb, hkv, bs, d, pool)
        dkp, dvp = to_torch(kp), to_torch(vp)
        q_out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
        for status in (torch.zeros(1, dtype=torch.int32, device="cuda"), None):
            pa.pa_rope_and_cache(q_out, dq, dk, dv, torch.tensor(pos, dtype=torch.int32, device="cuda"), to_torch(table), dkp,
                                 dvp, torch.tensor(slots, device="cuda"), status=status)
            if status is not None:
                assert status.item() == flag
        good = np.array([0, 2, 3, 4])
        sl, po = np.array(slots)[good], np.array(pos)[good]
        _oracle_append(pool, kp, vp, kv4.rotate_f32(k[good], po, table, False), kv4.widen32(v[good]), sl, bs, 1.0, 1.0)
        assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
        assert not to_numpy(q_out)[1].any() and to_numpy(q_out)[good].any()


def test_rope_special_values():
    """Infinities and NaN go through the formula; a NaN makes its 4-bit group NaN and touches no other."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs = 3, 1, 64, 16
    k = np.ones((n, hkv, d), np.float32)
    k[0, 0, 3], k[1, 0, 40] = np.nan, np.inf
    v = k.copy()
    table = kv4.cos_sin_table(8, d)
    kp = np.zeros((1, hkv, bs * 36), np.uint8)
    vp = kp.copy()
    dkp, dvp = to_torch(kp), to_torch(vp)
    pos, slots = np.array([1, 2, 3], np.int32), np.array([0, 5, 15], np.int64)
    pa.pa_rope_and_cache(None, None, to_torch(k), to_torch(v), to_torch(pos), to_torch(table), dkp, dvp, to_torch(slots))
    with np.errstate(invalid="ignore"):
        kv4.append_fp4(kv4.rotate_f32(k, pos, table, False), v, kp, vp, slots, bs, 1.0, 1.0)
    assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
    got = kv4.values(to_numpy(dvp), d, bs)
    assert np.isnan(got[0, 0, 0, :16]).all() and np.isfinite(got[0, 0, 0, 16:]).all() and np.isfinite(got[0, 0, 5]).all()


@pytest.mark.parametrize("scale", [0.043, 2.0 ** -5, 1e30, 3e-33])
def test_rope_fp8_codes_of_any_bits(scale):
    """Values (not turned) quantised over the whole range of fp32."""
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs, nb = 40, 2, 128, 16, 4
    rng = np.random.default_rng(5)
    bits = rng.integers(0, 1 << 32, (n, hkv, d), dtype=np.uint32)
    near = (rng.standard_normal((n, hkv, d)) * np.exp2(rng.integers(-12, 10, (n, hkv, d))) * np.float64(np.float32(scale)))
    with np.errstate(over="ignore"):
        near = np.clip(near, -3e38, 3e38).astype(np.float32).view(np.uint32)
    v = np.where(rng.random((n, hkv, d)) < 0.8, near, bits).astype(np.uint32).view(np.float32)
    v[np.isnan(v)] = np.nan  # one NaN pattern: the code is the NaN code either way
    v[:, :, 5] = -0.0
    k = np.ones((n, hkv, d), np.float32)
    table = kv4.cos_sin_table(4, d)
    slots, pos = np.arange(n, dtype=np.int64), np.zeros(n, np.int32)
    kp, vp = np.zeros((nb, hkv, bs, d), np.uint8), np.zeros((nb, hkv, bs, d), np.uint8)
    dkp, dvp = to_torch(kp), to_torch(vp)
    pa.pa_rope_and_cache(None, None, to_torch(k), to_torch(v), to_torch(pos), to_torch(table), dkp, dvp, to_torch(slots),
                         k_scale=1.0, v_scale=scale)
    with np.errstate(all="ignore"):
        want = oracle.e4m3_encode(v / np.float32(scale))
    got = to_numpy(dvp).transpose(0, 2, 1, 3).reshape(nb * bs, hkv, d)[:n]
    bad = np.isnan(v)
    assert np.all((got[bad] & 0x7F) == 0x7F) and np.array_equal(got[~bad], want[~bad])


def test_rope_on_another_stream_and_captured():
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 40, 8, 2, 128, 16, 6
    _, (dq, dk, dv) = _inputs(8, n, hq, hkv, d, "bf16", True)
    table = to_torch(kv4.cos_sin_table(MAXP, d))
    pos, slots = to_torch(np.arange(n, dtype=np.int32)), to_torch(np.arange(n, dtype=np.int64))
    new = lambda: [torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")] + [  # noqa: E731
        torch.zeros(nb, hkv, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    a, b, c = new(), new(), new()
    pa.pa_rope_and_cache(a[0], dq, dk, dv, pos, table, a[1], a[2], slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_and_cache(b[0], dq, dk, dv, pos, table, b[1], b[2], slots, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rope_and_cache(c[0], dq, dk, dv, pos, table, c[1], c[2], slots)
    graph.replay()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)
    dq.mul_(-1)  # a replay reads the buffers anew
    pa.pa_rope_and_cache(a[0], dq, dk, dv, pos, table, a[1], a[2], slots)
    graph.replay()
    assert torch.equal(a[0], c[0])
