"""GPU: the 4-bit kernels' forms that only some calls reach, and quotients beside the codes' borders."""
import numpy as np
import pytest

import oracle
import synth
from gpu_cases import status_word, to_numpy, to_torch
from oracle import kv4
from test_gpu_fp4 import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,bs,seqs,part", [
    (8, 1, 128, 32, 2400, 0), (16, 2, 128, 32, 2300, 64), (1, 1, 128, 16, 9700, 0), (8, 1, 64, 16, 15700, 0), (8, 1, 64, 32, 15700, 0),
    (8, 1, 64, 16, 10500, 32), (4, 1, 64, 32, 13000, 64)])
def test_decode_of_batches_past_the_16_warp_kernel(hq, hkv, d, bs, seqs, part):
    """So many sequences that their lengths leave no room for 16 warps' rings: 8 warps a CTA."""
    import paged_kv_cache_280_gb300 as pa

    lens = synth.uniform_ints(78, seqs, 0, 20).astype(np.int32)
    lens[seqs // 3], lens[seqs - 2] = 700, 90
    c = Case(25 + d + bs, hq, hkv, d, bs, lens)
    smem = pa.pa_decode_launch_info(seqs, hq, hkv, d, bs, c.tables.shape[1], pa.PA_FP4_E2M1, part)[2]
    rings = 16 * 2 * 2 * 32 * (d // 2 + d // 16)  # 16 warps, 2 stages of 32 tokens, K and V
    slots = 16 * (hq // hkv * (d + 2) * 4)
    assert rings + slots + seqs * (12 if part else 8) > 227 * 1024 >= smem
    at = [0, 1, 2, seqs // 3 - 1, seqs // 3, seqs // 3 + 1, seqs - 3, seqs - 2, seqs - 1] + list(range(50, seqs, seqs // 40))
    got = c.run(part)
    assert status_word(c.ws) == 0 and not np.any(got[lens == 0])
    c.check(got, seqs=at)


def _beside(x, rng):
    """Values up to three steps of fp32 from x."""
    x = x.astype(np.float32)
    k = rng.integers(-3, 4, x.shape)
    for _ in range(3):
        x = np.where(k > 0, np.nextafter(x, np.float32(np.inf)), np.where(k < 0, np.nextafter(x, np.float32(-np.inf)), x))
        k -= np.sign(k)
    return x


SCALES = np.exp2(np.random.default_rng(7).uniform(-16, 16, 40)).astype(np.float32)
SCALES[:4] = [1 + 2.0 ** -23, 2 - 2.0 ** -23, 4 / 3, 1.5]


def test_4_bit_codes_beside_their_borders():
    """Elements within three steps of fp32 of a border between two codes, and group maxima beside a border between two
    scales, for pool scales of any significand."""
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs, nb = 64, 2, 128, 32, 3
    e4m3 = oracle.e4m3_value(np.arange(127, dtype=np.uint8)).astype(np.float64)
    borders = (kv4.MAGNITUDES[1:] + kv4.MAGNITUDES[:-1]) / 2
    slots = np.arange(n, dtype=np.int64)
    for i, b in enumerate(SCALES):
        rng = np.random.default_rng(i)
        x = np.zeros((2, n, hkv, d // 16, 16), np.float32)
        j = rng.integers(1, 126, x.shape[:-1])
        s = e4m3[j]
        top = np.where(rng.random(s.shape) < 0.5, s, (e4m3[j] + e4m3[j + 1]) / 2)  # a scale, or the border above it
        x[...] = _beside(rng.choice(borders, x.shape) * s[..., None] * np.float64(b), rng) * rng.choice([-1, 1], x.shape)
        x[..., 5] = _beside(6 * top * np.float64(b), rng)
        x = x.reshape(2, n, hkv, d)
        kp, vp = (np.zeros((nb, hkv, bs * (d // 2 + d // 16)), np.uint8) for _ in range(2))
        dk, dv = to_torch(kp), to_torch(vp)
        pa.pa_reshape_and_cache_fp4(to_torch(x[0]), to_torch(x[1]), dk, dv, to_torch(slots), float(b), float(b))
        kv4.append_fp4(x[0], x[1], kp, vp, slots, bs, b, b)
        assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp), b


def test_fp8_codes_beside_their_borders():
    """The rotating append's FP8 values within three steps of fp32 of a border between two codes."""
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs, nb = 64, 2, 128, 32, 2
    e4m3 = oracle.e4m3_value(np.arange(127, dtype=np.uint8)).astype(np.float64)
    borders = (e4m3[1:] + e4m3[:-1]) / 2
    slots, pos = np.arange(n, dtype=np.int64), np.zeros(n, np.int32)
    table = to_torch(kv4.cos_sin_table(4, d))
    k = to_torch(np.zeros((n, hkv, d), np.float32))
    for i, b in enumerate(SCALES):
        rng = np.random.default_rng(i)
        v = (_beside(rng.choice(borders, (n, hkv, d)) * np.float64(b), rng) * rng.choice([-1, 1], (n, hkv, d))).astype(np.float32)
        kp, vp = (to_torch(np.zeros((nb, hkv, bs, d), np.uint8)) for _ in range(2))
        pa.pa_rope_and_cache(None, None, k, to_torch(v), to_torch(pos), table, kp, vp, to_torch(slots), k_scale=1.0, v_scale=float(b))
        want = oracle.e4m3_encode(v / b)
        assert np.array_equal(to_numpy(vp).transpose(0, 2, 1, 3).reshape(nb * bs, hkv, d), want), b


def test_nothing_to_append_or_unpack():
    import torch
    import paged_kv_cache_280_gb300 as pa

    d, hkv, bs = 64, 2, 16
    kp, vp = (torch.full((3, hkv, bs * 36), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
    none = torch.empty(0, hkv, d, device="cuda")
    slots, ids = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_fp4(none, none, kp, vp, slots, 1.0, 1.0, status=status)
    pa.pa_rope_and_cache(none, none, none, none, ids, torch.ones(4, d, device="cuda"), kp, vp, slots, status=status)
    out = torch.empty(0, hkv, bs, d, device="cuda")
    pa.pa_unpack_blocks_fp4(kp, vp, ids, out, out, 1.0, 1.0, status=status)
    assert status.item() == 0 and (kp == 9).all() and (vp == 9).all()


def test_rows_and_outputs_past_32_bits():
    """Inputs and outputs of more than 2^32 bytes and 2^31 elements: the last tokens, behind padding, and the last blocks."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, heads, d, bs, nb, last = 150_000, 128, 128, 32, 2, 20
    x = torch.zeros(n, heads, d, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 31
    rows = synth.normal(synth.stream_seed(61, 1), last * heads * d, "bf16").reshape(last, heads, d)
    x[-last:] = to_torch(rows)
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    at = np.arange(last) + 7
    slots[-last:] = to_torch(at)
    pools = [torch.zeros(nb, heads, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pa.pa_reshape_and_cache_fp4(x, x, *pools, slots, 0.5, 2.0)
    kp, vp = (np.zeros((nb, heads, bs * 72), np.uint8) for _ in range(2))
    kv4.append_fp4(rows, rows, kp, vp, at, bs, 0.5, 2.0)
    assert np.array_equal(to_numpy(pools[0]), kp) and np.array_equal(to_numpy(pools[1]), vp)

    # queries and keys and values as parts of the same rows
    hq, hkv = 64, 32
    table = kv4.cos_sin_table(64, d)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[-last:] = 9
    q_out = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    pools = [torch.zeros(nb, hkv, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2)]
    pa.pa_rope_and_cache(q_out, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, to_torch(table), *pools, slots, k_scale=0.5,
                         v_scale=2.0)
    kp, vp = (np.zeros((nb, hkv, bs * 72), np.uint8) for _ in range(2))
    p9 = np.full(last, 9)
    kv4.append_fp4(kv4.rotate_f32(rows[:, hq:hq + hkv], p9, table, False), kv4.widen32(rows[:, hq + hkv:]), kp, vp, at, bs, 0.5, 2.0)
    assert np.array_equal(to_numpy(pools[0]), kp) and np.array_equal(to_numpy(pools[1]), vp)
    assert np.array_equal(to_numpy(q_out[-last:]), kv4.to_bf16(kv4.rotate_f32(rows[:, :hq], p9, table, False)))
    assert not q_out[:-last].any()
    del x, q_out

    num, hkv = 5_000, 128
    pools = [torch.randint(0x20, 0x41, (3, hkv, bs * 72), device="cuda", dtype=torch.uint8) for _ in range(2)]
    ids = (torch.arange(num, device="cuda", dtype=torch.int32) + 1) % 3
    out = [torch.empty(num, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert out[0].numel() > 1 << 31
    pa.pa_unpack_blocks_fp4(*pools, ids, *out, 1.0, 0.25)
    for o, p, s in zip(out, pools, (1.0, 0.25)):
        for i in (0, num // 2, num - 2, num - 1):
            want = kv4.to_bf16(kv4.values(to_numpy(p)[[int(ids[i])]], d, bs).astype(np.float32) * np.float32(s))
            assert np.array_equal(to_numpy(o[[i]]), want)
