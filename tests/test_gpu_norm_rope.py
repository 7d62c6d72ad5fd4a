"""GPU: the normed rotating append (pa_norm_rope_and_cache) against the definition in float64, into every pool type."""
import numpy as np
import pytest

import oracle
import synth
from gpu_cases import to_numpy, to_torch, widen
from oracle import chunks, kv4
from test_gpu_rope import MAXP, _inputs, _pool

pytestmark = pytest.mark.gpu

EPS = 1e-6

CASES = [
    # n, hq, hkv, d, bs, in, pool, rot, interleaved, fused
    (1, 8, 2, 128, 16, "bf16", "bf16", 128, False, True),
    (1, 1, 1, 64, 32, "f32", "f32", 64, True, False),
    (37, 32, 8, 128, 16, "bf16", "bf16", 128, False, True),
    (37, 5, 5, 64, 32, "bf16", "bf16", 32, False, False),
    (37, 6, 3, 128, 32, "bf16", "bf16", 48, True, True),
    (23, 7, 1, 128, 16, "f32", "f32", 16, False, True),
    (23, 4, 4, 64, 16, "f32", "f32", 64, True, False),
    (31, 8, 8, 128, 16, "bf16", "fp8", 128, False, True),
    (31, 16, 2, 128, 32, "f32", "fp8", 64, True, False),
    (33, 3, 3, 64, 32, "bf16", "fp4", 32, False, True),
    (33, 12, 4, 128, 32, "f32", "fp4", 96, False, True),
    (700, 32, 8, 128, 16, "bf16", "fp4", 128, False, True),  # more rows than one turn of the grid
    (2000, 16, 8, 64, 16, "f32", "f32", 64, False, False),
]


def _want(x, w, pos, table, inter):
    """(the definition in float64, a bound on the fp32 error before the last rounding)."""
    y = chunks.head_norm(x, w, EPS)
    turned = kv4._rotate(y, pos, table.astype(np.float64), inter)
    # the squares' sum (D + 1 roundings), its root (one, and half of the sum's), two products: D / 2 + 4 units of 2^-24;
    # the rotation: two products and a sum of two elements no larger than the row's largest
    d = x.shape[-1]
    size = np.abs(y).max(-1, keepdims=True)
    return turned, ((d / 2 + 4) * 2 + 3 * 2) * 2.0 ** -24 * size


def _near(got, want, slack, half):
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= slack + half * (np.abs(want) + slack)), f"max |err| {err.max():.3e}"


def _pool_rows(pool, kind, slots, bs, d, scale):
    """float64 [N][Hkv][D] that the pool holds at the slots."""
    if kind in ("fp8", "fp4"):
        v = chunks.pool_values(pool, kind, d, bs) * np.float64(np.float32(scale))
    else:
        v = widen(pool)
    return v[slots // bs, :, slots % bs]


def _check_stored(got, want, slack, kind, scale):
    """A stored value against the definition: within the storing's rounding of some value that is within slack."""
    if kind == "bf16":
        _near(got, want, slack, 2.0 ** -8)
    elif kind == "f32":
        _near(got, want, slack, 2.0 ** -24)
    elif kind == "fp8":  # half a step: 2^-4 of the value, 2^-10 of the pool scale among the smallest; saturated at 448
        a = np.clip(want, -448 * scale, 448 * scale)
        assert np.all(np.abs(got - a) <= 2.0 ** -4 * (np.abs(a) + slack) + 2.0 ** -10 * scale + slack)
    else:
        # the scale is off by 2^-4 of itself at most (2^-10 of the pool scale among the smallest), so a code's value is off by a
        # quarter of the largest at most between 4 and 6 (half a step of 2, of 6), and one sixteenth for the scale; the largest
        # may saturate by a sixteenth
        g = np.abs(want).reshape(*want.shape[:-1], -1, 16).max(-1)
        g = np.repeat(g, 16, -1)
        assert np.all(np.abs(got - want) <= (1 / 6 + 1 / 16) * (1 + 1 / 16) * (g + slack) + 2.0 ** -10 * 6 * scale + slack)


@pytest.mark.parametrize("n,hq,hkv,d,bs,dtype,pool,rot,inter,fused", CASES)
def test_norm_rope(n, hq, hkv, d, bs, dtype, pool, rot, inter, fused):
    import torch
    import paged_kv_cache_280_gb300 as pa

    seed = 3000 + n + hq + d + rot
    (q, k, v), (dq, dk, dv) = _inputs(seed, n, hq, hkv, d, dtype, fused)
    nb = -(-n // bs) + 3
    slots = synth.permutation(seed, nb * bs)[:n].astype(np.int64)
    if n > 5:
        slots[[2, n - 1]] = -1  # padding
    pos = synth.uniform_ints(seed + 1, n, 0, MAXP - 1).astype(np.int32)
    pos[0] = MAXP - 1
    if n > 5:
        pos[2] = -5  # a padding token's position is not looked at
    rng = np.random.default_rng(seed)
    qw, kw = (rng.uniform(0.25, 2, d).astype(np.float32) * rng.choice([-1, 1], d).astype(np.float32) for _ in range(2))
    table = kv4.cos_sin_table(MAXP, rot)
    kp, vp = _pool(seed, nb, hkv, bs, d, pool), _pool(seed + 7, nb, hkv, bs, d, pool)
    dkp, dvp = to_torch(kp), to_torch(vp)
    ks, vs = 0.037, 1.75
    q_out, k_out = (to_torch(_pool(3, n, h, 1, d, dtype).reshape(n, h, d)) for h in (hq, hkv))
    q_before, k_before = widen(to_numpy(q_out)).copy(), widen(to_numpy(k_out)).copy()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (dq, dk, dv, to_torch(qw), to_torch(kw), EPS, to_torch(pos), to_torch(table))
    pa.pa_norm_rope_and_cache(q_out, k_out, *args, dkp, dvp, to_torch(slots), interleaved=inter, k_scale=ks, v_scale=vs,
                              status=status)
    assert status.item() == 0
    kept = slots >= 0
    safe = np.where(kept, pos, 0)
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    (wq, sq), (wk, sk) = _want(q, qw, safe, table, inter), _want(k, kw, safe, table, inter)
    for got, want, slack, before in ((q_out, wq, sq, q_before), (k_out, wk, sk, k_before)):
        got = widen(to_numpy(got))
        _near(got[kept], want[kept], slack[kept], half)
        assert np.array_equal(got[~kept], before[~kept])
    _check_stored(_pool_rows(to_numpy(dkp), pool, slots[kept], bs, d, ks), wk[kept], sk[kept], pool, np.float64(np.float32(ks)))
    # values are stored as pa_rope_and_cache stores them, bit for bit, and nothing else of the pools changes
    k2, v2 = to_torch(kp), to_torch(vp)
    pa.pa_rope_and_cache(None, None, dk, dv, to_torch(pos), to_torch(table), k2, v2, to_torch(slots), interleaved=inter,
                         k_scale=ks, v_scale=vs)
    assert torch.equal(dvp, v2)
    untouched = np.setdiff1d(np.arange(nb * bs), slots[kept])
    if pool != "fp4":
        a, b = to_numpy(dkp).transpose(0, 2, 1, 3), kp.transpose(0, 2, 1, 3)
        assert np.array_equal(a.reshape(nb * bs, hkv, d)[untouched], b.reshape(nb * bs, hkv, d)[untouched])
    else:
        for a, b in zip(kv4.split(to_numpy(dkp), d, bs), kv4.split(kp, d, bs)):
            a, b = (t.transpose(0, 2, 1, 3).reshape(nb * bs, -1) for t in (a, b))
            assert np.array_equal(a[untouched], b[untouched])
    # the turned keys, stored from k_out's bits, give the same pool where both round to in_dtype
    if pool == dtype:
        rows = to_numpy(dkp)[slots[kept] // bs, :, slots[kept] % bs]
        assert np.array_equal(rows, to_numpy(k_out)[kept])


def test_norm_rope_in_place_and_without_queries():
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 19, 8, 2, 128, 16, 4
    _, (dq, dk, dv) = _inputs(5, n, hq, hkv, d, "bf16", False)
    slots, pos = to_torch(np.arange(n, dtype=np.int64) + 3), to_torch(np.arange(n, dtype=np.int32))
    table = to_torch(kv4.cos_sin_table(MAXP, d))
    w = torch.linspace(0.5, 2, d, device="cuda")
    pools = [torch.zeros(nb, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    q2, k2 = torch.empty_like(dq), torch.empty_like(dk)
    pa.pa_norm_rope_and_cache(q2, k2, dq, dk, dv, w, w, EPS, pos, table, pools[0], pools[1], slots)
    pa.pa_norm_rope_and_cache(None, None, None, dk, dv, None, w, EPS, pos, table, pools[2], pools[3], slots)
    pa.pa_norm_rope_and_cache(dq, dk, dq, dk, dv, w, w, EPS, pos, table, pools[4], pools[5], slots)
    assert torch.equal(dq, q2) and torch.equal(dk, k2)
    for i in (2, 4):
        assert torch.equal(pools[0], pools[i]) and torch.equal(pools[1], pools[i + 1])


@pytest.mark.parametrize("pool", ["bf16", "fp8"])
def test_norm_rope_flags_bad_slots_and_positions(pool):
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 5, 4, 2, 128, 16, 3
    _, (dq, dk, dv) = _inputs(6, n, hq, hkv, d, "bf16", True)
    table, w = to_torch(kv4.cos_sin_table(MAXP, d)), torch.ones(d, device="cuda")
    for slots, pos, flag in (([1, nb * bs, 3, 4, 5], [1, 2, 3, 4, 5], pa.PA_DEV_BAD_SLOT),
                             ([1, 2, 3, 4, 5], [1, MAXP, 3, 4, 5], pa.PA_DEV_BAD_POSITION),
                             ([1, 1 << 40, 3, 4, 5], [1, -1, 3, 4, 5], pa.PA_DEV_BAD_SLOT | pa.PA_DEV_BAD_POSITION)):
        kp, vp = (to_torch(_pool(i, nb, hkv, bs, d, pool)) for i in (1, 2))
        before = [kp.clone(), vp.clone()]
        q_out, k_out = (torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_norm_rope_and_cache(q_out, k_out, dq, dk, dv, w, w, EPS, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                                  table, kp, vp, torch.tensor(slots, device="cuda"), status=status)
        assert status.item() == flag
        good = [0, 2, 3, 4]
        assert not q_out[1].any() and not k_out[1].any() and q_out[good].any(-1).all() and k_out[good].any(-1).all()
        at = [slots[i] for i in good]
        rows = [p.transpose(1, 2).reshape(nb * bs, hkv, d) for p in (kp, vp, *before)]
        rest = [i for i in range(nb * bs) if i not in at]
        assert torch.equal(rows[0][rest], rows[2][rest]) and torch.equal(rows[1][rest], rows[3][rest])


def test_norm_rope_special_rows():
    """A row of zeros stays zero; a NaN or an infinity makes its own head NaN and no other; a row whose squares leave fp32 is zero."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs = 5, 2, 64, 16
    k = torch.ones(n, hkv, d, device="cuda")
    k[0, 0], k[1, 0, 3], k[2, 1, 40], k[3, 0] = 0, float("nan"), float("inf"), 3e38
    k[4, 1] = 1e-30
    v = torch.zeros_like(k)
    pool = torch.zeros(1, hkv, bs, d, device="cuda")
    k_out = torch.empty_like(k)
    table, w = to_torch(kv4.cos_sin_table(8, d)), torch.full((d,), 2.0, device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")  # no turn
    pa.pa_norm_rope_and_cache(None, k_out, None, k, v, None, w, EPS, pos, table, pool, pool.clone(), torch.arange(n, device="cuda"))
    assert not k_out[0, 0].any() and not k_out[3, 0].any() and (k_out[4, 1].abs() < 1e-26).all()
    assert k_out[1, 0].isnan().any() and k_out[2, 1].isnan().any()
    ok = torch.tensor([[1, 1], [0, 1], [1, 0], [1, 1], [1, 1]], dtype=torch.bool, device="cuda")
    assert k_out[ok].isfinite().all()
    assert torch.allclose(k_out[0, 1], torch.full((d,), 2.0, device="cuda"), rtol=1e-6)


def test_norm_rope_on_another_stream_and_captured():
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hq, hkv, d, bs, nb = 40, 8, 2, 128, 16, 6
    _, (dq, dk, dv) = _inputs(8, n, hq, hkv, d, "bf16", True)
    table, w = to_torch(kv4.cos_sin_table(MAXP, d)), torch.linspace(0.5, 2, d, device="cuda")
    pos, slots = to_torch(np.arange(n, dtype=np.int32)), to_torch(np.arange(n, dtype=np.int64))
    new = lambda: [torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv)] + [  # noqa: E731
        torch.zeros(nb, hkv, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    call = lambda x, **kw: pa.pa_norm_rope_and_cache(x[0], x[1], dq, dk, dv, w, w, EPS, pos, table, x[2], x[3], slots, **kw)  # noqa: E731
    a, b, c = new(), new(), new()
    call(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(b, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c)
    graph.replay()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)
    dq.mul_(-1)  # a replay reads the buffers anew
    call(a)
    graph.replay()
    assert torch.equal(a[0], c[0])


@pytest.mark.parametrize("case", [(3000, 24, 8, 128, 16, "bf16", "fp8", 128, False, True),
                                  (4000, 40, 16, 64, 32, "f32", "fp4", 32, True, False),
                                  (5003, 15, 5, 128, 16, "bf16", "bf16", 64, False, True)])
def test_norm_rope_rows_behind_one_another(case):
    """Several rows to a thread, across tokens and from keys to values, with padding among them."""
    test_norm_rope(*case)
