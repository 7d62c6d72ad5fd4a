"""GPU: appends of several turns of their grids, where rows, slots and positions are fetched turns ahead -- a call of four turns
and more against calls of less than one turn each and, on some of its tokens, against the oracle."""
import numpy as np
import pytest

import oracle
from gpu_cases import to_numpy, to_torch
from oracle import kv4

pytestmark = pytest.mark.gpu

MAXP = 5000


def _torch_dtype(name):
    import torch

    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _pools(seed, nb, hkv, bs, d, pool):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    if pool in ("fp4", "fp8"):
        shape = (nb, hkv, bs * (d // 2 + d // 16)) if pool == "fp4" else (nb, hkv, bs, d)
        return [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    return [torch.randn((nb, hkv, bs, d), generator=g, device="cuda").to(_torch_dtype(pool)) for _ in range(2)]


def _rows(pool_tensor, kind, slots, d, bs):
    """What a pool holds at slots, as tensors whose first axis is the slots'."""
    blk, off = slots // bs, slots % bs
    if kind != "fp4":
        return (pool_tensor[blk, :, off],)
    nb, hkv, _ = pool_tensor.shape
    cut = bs * d // 2
    return (pool_tensor[..., :cut].reshape(nb, hkv, bs, d // 2)[blk, :, off],
            pool_tensor[..., cut:].reshape(nb, hkv, bs, d // 16)[blk, :, off])


def _slots(g, n, bs, per_turn):
    """Scattered slots; padding in every turn, slots past the pool in the later ones."""
    import torch

    nb = -(-n // bs) + 5
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:n]
    slots[torch.randperm(n, generator=g, device="cuda")[: n // 9]] = -1
    slots[3 * per_turn + 1::per_turn // 3 + 1] = nb * bs + 7
    return nb, slots


def _sample(n, per_turn, slots, limit):
    """Tokens to look at closely: around the ends of the turns, the last ones, and some anywhere, that are written."""
    at = np.concatenate([np.arange(t * per_turn - 3, t * per_turn + 4) for t in range(1, n // per_turn + 1)] +
                        [np.arange(0, 4), np.arange(n - 9, n), np.random.default_rng(n).integers(0, n, 40)])
    at = np.unique(at[(at >= 0) & (at < n)])
    s = to_numpy(slots)[at]
    return at[(s >= 0) & (s < limit)]


@pytest.mark.parametrize("dtype,pool,hq,hkv,d,bs,rot,inter,in_place", [
    ("bf16", "bf16", 32, 8, 128, 16, 128, False, False), ("bf16", "bf16", 7, 7, 64, 32, 32, True, True),
    ("f32", "f32", 9, 3, 128, 32, 96, False, True), ("f32", "f32", 16, 4, 64, 16, 64, True, False),
    ("bf16", "fp8", 12, 4, 128, 16, 128, False, True), ("f32", "fp8", 5, 5, 128, 32, 64, True, False),
    ("bf16", "fp4", 32, 8, 128, 16, 128, False, False), ("f32", "fp4", 3, 3, 64, 32, 32, True, True),
    ("bf16", "fp4", 0, 5, 64, 16, 64, False, False)])
def test_rotating_append(dtype, pool, hq, hkv, d, bs, rot, inter, in_place):
    import torch
    import paged_kv_cache_280_gb300 as pa

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads = hq + 2 * hkv
    per_turn = sms * 4 * 256 // (heads * (d // 16))  # tokens of one turn of a grid of four CTAs of 256 threads per SM
    n = int(4.3 * per_turn) + 1
    g = torch.Generator(device="cuda").manual_seed(n)
    qkv = torch.randn((n, heads, d), generator=g, device="cuda").to(_torch_dtype(dtype))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    nb, slots = _slots(g, n, bs, per_turn)
    pos = torch.randint(0, MAXP, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[per_turn // 2::per_turn // 2 + 5] = MAXP  # out of range, in every turn
    host_table = kv4.cos_sin_table(MAXP, rot)
    table = to_torch(host_table)
    ks, vs = 0.037, 2.0

    def run(step):
        pools = _pools(n, nb, hkv, bs, d, pool)
        qs = q.clone() if in_place else q
        out = qs if in_place else torch.full((n, hq, d), 7.0, device="cuda", dtype=q.dtype)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for a in range(0, n, step):
            s = slice(a, a + step)
            pa.pa_rope_and_cache(out[s] if hq else None, qs[s] if hq else None, k[s], v[s], pos[s], table, *pools, slots[s],
                                 interleaved=inter, k_scale=ks, v_scale=vs, status=status)
        assert status.item() == pa.PA_DEV_BAD_SLOT | pa.PA_DEV_BAD_POSITION
        return [out, *pools]

    whole, parts = run(n), run(per_turn * 2 // 3)
    for a, b in zip(whole, parts):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    at = _sample(n, per_turn, slots, nb * bs)
    at = at[to_numpy(pos)[at] < MAXP]
    assert len(at) > 30
    dat = torch.from_numpy(at).cuda()
    hpos = to_numpy(pos)[at]
    if hq:
        want = kv4.rotate_f32(to_numpy(q[dat]), hpos, host_table, inter)
        assert np.array_equal(to_numpy(whole[0][dat]), want if dtype == "f32" else kv4.to_bf16(want))
        kept = to_numpy(whole[0][(slots < 0)][:5]), to_numpy((q if in_place else torch.full_like(q, 7.0))[(slots < 0)][:5])
        assert np.array_equal(*kept)  # padding
    rk, rv = kv4.rotate_f32(to_numpy(k[dat]), hpos, host_table, inter), kv4.widen32(to_numpy(v[dat]))
    for x, dev, scale in ((rk, whole[1], ks), (rv, whole[2], vs)):
        got = [to_numpy(r) for r in _rows(dev, pool, slots[dat], d, bs)]
        want = kv4.quantise_rows(x, scale) if pool == "fp4" else \
            (oracle.e4m3_encode(x / np.float32(scale)),) if pool == "fp8" else (x if pool == "f32" else kv4.to_bf16(x),)
        assert all(np.array_equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype,hkv,d,bs", [("bf16", 8, 128, 16), ("bf16", 3, 64, 32), ("f32", 8, 64, 16), ("f32", 5, 128, 32)])
def test_4_bit_append(dtype, hkv, d, bs):
    import torch
    import paged_kv_cache_280_gb300 as pa

    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_turn = sms * 2 * 256 // (hkv * (d // 16))  # tokens of one turn of the half of a grid of four CTAs per SM
    n = int(4.3 * per_turn) + 1
    g = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn((n, hkv, d), generator=g, device="cuda").to(_torch_dtype(dtype)) for _ in range(2))
    nb, slots = _slots(g, n, bs, per_turn)
    scales = 0.043, 0.5

    def run(step):
        pools = _pools(n, nb, hkv, bs, d, "fp4")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        for a in range(0, n, step):
            s = slice(a, a + step)
            pa.pa_reshape_and_cache_fp4(k[s], v[s], *pools, slots[s], *scales, status=status)
        assert status.item() == pa.PA_DEV_BAD_SLOT
        return pools

    whole, parts = run(n), run(per_turn * 2 // 3)
    for a, b in zip(whole, parts):
        assert torch.equal(a, b)
    at = _sample(n, per_turn, slots, nb * bs)
    assert len(at) > 30
    dat = torch.from_numpy(at).cuda()
    for x, dev, scale in ((k, whole[0], scales[0]), (v, whole[1], scales[1])):
        want = kv4.quantise_rows(kv4.widen32(to_numpy(x[dat])), scale)
        assert all(np.array_equal(to_numpy(a), b) for a, b in zip(_rows(dev, "fp4", slots[dat], d, bs), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
def test_unpacking_to_outputs_that_are_16_byte_aligned_only(d, bs, dtype):
    import torch
    import paged_kv_cache_280_gb300 as pa

    nb, hkv, n, ks, vs = 30, 3, 17, 0.37, 1 / 128
    kp, vp = _pools(d + bs, nb, hkv, bs, d, "fp4")
    blocks = torch.randperm(nb, device="cuda")[:n].to(torch.int32)
    t = _torch_dtype(dtype)
    shift = 16 // t.itemsize

    def run(off):
        flat = [torch.zeros(off + n * hkv * bs * d, dtype=t, device="cuda") for _ in range(2)]
        out = [f[off:].view(n, hkv, bs, d) for f in flat]
        pa.pa_unpack_blocks_fp4(kp, vp, blocks, *out, ks, vs)
        assert all(not f[:off].any() for f in flat)
        return out

    aligned, shifted = run(0), run(shift)
    assert aligned[0].data_ptr() % 32 == 0 and shifted[0].data_ptr() % 32 == 16
    for a, b, pool, scale in zip(aligned, shifted, (kp, vp), (ks, vs)):
        assert torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))
        want = kv4.values(to_numpy(pool[blocks.long()]), d, bs).astype(np.float32) * np.float32(scale)
        bad = np.isnan(want)
        want = want if dtype == "f32" else kv4.to_bf16(want)
        assert np.array_equal(to_numpy(b)[~bad], want[~bad])
