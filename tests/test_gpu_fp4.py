"""GPU: 4-bit pools -- append and unpacking bit-exact against the oracle, decode within a derived bound of float64,
whole-block copies, and the chains in which a serving step uses them."""
import numpy as np
import pytest

import oracle
import synth
from gpu_cases import status_word, to_numpy, to_torch, widen
from oracle import kv4

pytestmark = pytest.mark.gpu


def _random_pool(seed, nb, hkv, bs, d):
    """Any codes; scales between 2^-3 and 2."""
    r = np.random.default_rng(seed)
    p = r.integers(0, 256, (nb, hkv, bs * (d // 2 + d // 16))).astype(np.uint8)
    p[..., bs * d // 2:] = r.integers(0x20, 0x41, p[..., bs * d // 2:].shape)
    return p


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hkv,d,bs,scales", [(1, 1, 64, 16, (1.0, 1.0)), (37, 4, 128, 16, (0.037, 2.5)),
                                               (300, 3, 64, 32, (0.3, 0.011)), (129, 8, 128, 32, (1 / 64, 7.0))])
def test_append_bit_exact(n, hkv, d, bs, scales, dtype):
    import torch
    import paged_kv_cache_280_gb300 as pa

    rng = np.random.default_rng(n + d)
    x = rng.standard_normal((2, n, hkv, d)) * np.exp2(rng.integers(-12, 9, (2, n, hkv, d // 16))).repeat(16, -1)
    if n > 1:  # every code and every tie of a group whose scale is exact, both signs; zero, tiny, NaN, infinite groups
        grid = np.concatenate([kv4.MAGNITUDES, (kv4.MAGNITUDES[1:] + kv4.MAGNITUDES[:-1]) / 2, [6.0]])
        x[0, 0, 0, :16], x[1, 0, 0, :16] = grid * scales[0], -grid * scales[1]
        x[0, 1, 0, :16], x[0, 1, 0, 16:32], x[0, 1, 0, 32] = 0.0, 1e-7, np.nan
        x[1, 1, 0, 3], x[1, 1, 0, 17], x[1, 2, 0, :16] = np.inf, -np.inf, 1e30
    x = x.astype(np.float32)
    kn, vn = (x if dtype == "f32" else kv4.to_bf16(x))
    nb = -(-n // bs) + 2
    slots = synth.permutation(n, nb * bs)[:n].astype(np.int64)
    if n > 5:
        slots[3] = -1
    kp, vp = _random_pool(1, nb, hkv, bs, d), _random_pool(2, nb, hkv, bs, d)
    dk, dv = to_torch(kp), to_torch(vp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_fp4(to_torch(kn), to_torch(vn), dk, dv, to_torch(slots), *scales, status=status)
    kv4.append_fp4(kn, vn, kp, vp, slots, bs, *scales)
    assert status.item() == 0
    assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp)


@pytest.mark.parametrize("scale", [1.0, 0.043, 3.0 * 2.0 ** 59, 1.1 * 2.0 ** -60, 1e30, 3e-33, 1e-40, 2.0 ** -30])
def test_append_of_any_bits(scale):
    """Quotients over the whole range of fp32: every exponent, subnormal numbers and results, zeros of both signs,
    infinities and NaN, with pool scales in and out of the range where the quotients are formed by multiplication."""
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs, nb = 64, 4, 128, 16, 5
    rng = np.random.default_rng(17)
    bits = rng.integers(0, 1 << 32, (2, n, hkv, d), dtype=np.uint32)
    # half of the groups: elements near each other in size, around the pool scale and over fp32's range of it
    near = (rng.standard_normal((2, n, hkv, d)) * np.exp2(rng.integers(-14, 14, (2, n, hkv, d // 16))).repeat(16, -1)
            * np.float64(np.float32(scale)))
    with np.errstate(over="ignore"):
        near = np.clip(near, -3e38, 3e38).astype(np.float32).view(np.uint32)
    take = (rng.random((2, n, hkv, d // 16)) < 0.75).repeat(16, -1)
    bits = np.where(take, near, bits)
    bits[:, :, 0, ::7] = 0x80000000  # negative zeros
    kn, vn = bits.view(np.float32)
    slots = synth.permutation(3, nb * bs)[:n].astype(np.int64)
    kp, vp = _random_pool(1, nb, hkv, bs, d), _random_pool(2, nb, hkv, bs, d)
    dk, dv = to_torch(kp), to_torch(vp)
    pa.pa_reshape_and_cache_fp4(to_torch(kn), to_torch(vn), dk, dv, to_torch(slots), scale, scale)
    kv4.append_fp4(kn, vn, kp, vp, slots, bs, scale, scale)
    assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp)


def test_append_flags_a_bad_slot_and_leaves_the_rest():
    import torch
    import paged_kv_cache_280_gb300 as pa

    n, hkv, d, bs, nb = 3, 2, 64, 16, 2
    x = synth.normal(synth.stream_seed(4, 1), n * hkv * d, "bf16").reshape(n, hkv, d)
    kp, vp = _random_pool(1, nb, hkv, bs, d), _random_pool(2, nb, hkv, bs, d)
    dk, dv = to_torch(kp), to_torch(vp)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_reshape_and_cache_fp4(to_torch(x), to_torch(x), dk, dv, torch.tensor([4, nb * bs, 9], device="cuda"), 1.0, 1.0,
                                status=status)
    kv4.append_fp4(x[[0, 2]], x[[0, 2]], kp, vp, np.array([4, 9]), bs, 1.0, 1.0)
    assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp)
    assert status.item() == pa.PA_DEV_BAD_SLOT


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,hkv,d,bs", [(1, 1, 64, 16), (7, 3, 128, 16), (5, 2, 64, 32), (40, 8, 128, 32)])
def test_unpack_bit_exact(n, hkv, d, bs, dtype):
    import torch
    import paged_kv_cache_280_gb300 as pa

    nb, ks, vs = 50, 0.37, 1 / 128
    kp = np.random.default_rng(n).integers(0, 256, (nb, hkv, bs * (d // 2 + d // 16))).astype(np.uint8)  # NaN scales too
    vp = kp[::-1].copy()
    blocks = synth.permutation(n + 1, nb)[:n].astype(np.int32)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    out = [torch.zeros(n, hkv, bs, d, dtype=t, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_unpack_blocks_fp4(to_torch(kp), to_torch(vp), to_torch(blocks), *out, ks, vs, status=status)
    assert status.item() == 0
    for got, pool, scale in zip(out, (kp, vp), (ks, vs)):
        want = kv4.values(pool[blocks], d, bs).astype(np.float32) * np.float32(scale)
        got = to_numpy(got)
        bad = np.isnan(want)
        assert np.isnan(widen(got)[bad]).all()
        want = want if dtype == "f32" else kv4.to_bf16(want)
        assert np.array_equal(got[~bad], want[~bad])


def test_unpack_flags_a_bad_block_and_leaves_its_rows():
    import torch
    import paged_kv_cache_280_gb300 as pa

    hkv, d, bs, nb = 2, 128, 16, 4
    kp = _random_pool(1, nb, hkv, bs, d)
    for bad in (nb, -1):
        out = [torch.full((3, hkv, bs, d), 7.0, device="cuda") for _ in range(2)]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_unpack_blocks_fp4(to_torch(kp), to_torch(kp), torch.tensor([1, bad, 2], dtype=torch.int32, device="cuda"), *out, 1.0,
                                1.0, status=status)
        assert status.item() == pa.PA_DEV_BAD_BLOCK_ID
        for o in out:
            assert (o[1] == 7.0).all() and np.array_equal(to_numpy(o)[[0, 2]], kv4.values(kp[[1, 2]], d, bs).astype(np.float32))


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

class Case:
    def __init__(self, seed, hq, hkv, d, bs, lens, scales=(0.5, 0.25), q_size=1.0, extra_blocks=3):
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens // bs)
        self.nb = int(need.sum()) + extra_blocks
        order = synth.permutation(seed, self.nb).astype(np.int32)
        self.tables = np.zeros((len(lens), max(1, int(need.max()))), np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at: at + n]
            at += n
        self.kp, self.vp = _random_pool(seed, self.nb, hkv, bs, d), _random_pool(seed + 1, self.nb, hkv, bs, d)
        q = synth.normal(synth.stream_seed(seed, 3), len(lens) * hq * d, "f32").reshape(len(lens), hq, d)
        self.q = kv4.to_bf16(q * np.float32(q_size))
        self.scales, self.scale = scales, float(1 / np.sqrt(d) / q_size)
        # slots past each sequence's end, and free blocks, hold NaN scales and any codes
        used = np.zeros((self.nb, bs), bool)
        for b, n in enumerate(self.lens):
            for t in range(0, int(n), bs):
                used[self.tables[b, t // bs], : min(bs, n - t)] = True
        for p in (self.kp, self.vp):
            kv4.split(p, d, bs)[1].transpose(0, 2, 1, 3)[~used] = 0x7F
            cut = bs * d // 2
            s = p[..., cut:].reshape(self.nb, hkv, bs, d // 16)
            s.transpose(0, 2, 1, 3)[~used] = 0x7F
            p[..., cut:] = s.reshape(self.nb, hkv, -1)

    def run(self, part=0, plan=False, ws=None, tables=None, max_seq_len=None, stream=None):
        import torch
        import paged_kv_cache_280_gb300 as pa

        b = len(self.lens)
        self.dev = [to_torch(a) for a in (self.q, self.kp, self.vp, self.tables if tables is None else tables, self.lens)]
        q, kp, vp, tab, lens = self.dev
        out = torch.full_like(q, float("nan"))
        if ws is None:
            ws = torch.zeros(pa.pa_decode_workspace_bytes(b, self.hq, self.hkv, self.d), dtype=torch.uint8, device="cuda")
        msl = int(self.lens.max()) if max_seq_len is None else max_seq_len
        pl = None
        if plan:
            pl = to_torch(pa.pa_decode_build_plan(self.tables, self.lens, msl, self.hq, self.hkv, self.d, self.bs, part,
                                                  pa.PA_FP4_E2M1))
        pa.pa_decode_attention_fp4(out, q, kp, vp, *self.scales, tab, lens, msl, self.scale, ws, partition_tokens=part, plan=pl,
                                   stream=stream)
        torch.cuda.synchronize()
        self.ws = ws
        return to_numpy(out)

    def oracle(self, seqs=None):
        return kv4.decode_fp4(self.q, self.kp, self.vp, *self.scales, self.tables, self.lens, self.scale, self.bs, seqs)

    def check(self, got, seqs=None):
        """The output's own rounding to bf16 (2^-8) beside the oracle's bound."""
        ref, bound = self.oracle(seqs)
        rows = slice(None) if seqs is None else list(seqs)
        err, lim = np.abs(widen(got)[rows] - ref[rows]), 2.0 ** -8 * (np.abs(ref[rows]) + bound[rows]) + bound[rows]
        assert np.all(err <= lim), f"{np.max(err - lim):.3e} over the bound, at |ref| {np.abs(ref[rows]).max():.3g}"


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 250]


@pytest.mark.parametrize("hq,hkv,d,bs,part", [
    (8, 8, 128, 16, 0), (4, 2, 128, 32, 0), (32, 8, 128, 16, 0), (12, 4, 64, 16, 0), (8, 1, 64, 32, 0), (5, 1, 128, 16, 0),
    (14, 2, 128, 32, 0), (32, 4, 128, 16, 32), (16, 8, 64, 16, 64), (8, 8, 64, 32, 32), (1, 1, 64, 16, 0),
    (16, 16, 128, 16, 0), (48, 16, 64, 32, 0), (16, 16, 128, 32, 64)])  # the last three: more segments than CTAs
def test_decode_matches_oracle(hq, hkv, d, bs, part):
    c = Case(40 + hq + d + bs, hq, hkv, d, bs, LENS)
    got = c.run(part)
    assert status_word(c.ws) == 0
    assert not got[0].any()  # an empty sequence
    c.check(got)


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 8, 128, 16), (4, 4, 128, 32), (16, 2, 64, 16), (3, 3, 64, 32)])
def test_decode_merge_modes_and_plan(hq, hkv, d, bs, mode):
    """Split segments merged in the decode kernel and by the merge kernel; the host-built plan gives the same bits."""
    import paged_kv_cache_280_gb300 as pa

    c = Case(60 + hq + bs, hq, hkv, d, bs, [3000, 1, 0, 517, 1999, 64])
    try:
        pa.pa_debug_set_merge_mode(mode)
        got = c.run()
        c.check(got)
        assert np.array_equal(c.run(plan=True), got) and np.array_equal(c.run(ws=c.ws), got)
        assert status_word(c.ws) == 0
    finally:
        pa.pa_debug_set_merge_mode(0)


def test_launch_facts():
    import torch
    import paged_kv_cache_280_gb300 as pa

    ctas, stages, smem, mma = pa.pa_decode_launch_info(64, 32, 8, 128, 16, 256, pa.PA_FP4_E2M1)
    assert (ctas, stages, mma) == (torch.cuda.get_device_properties(0).multi_processor_count, 2, 1) and smem <= 227 * 1024
    assert pa.pa_decode_kernels_per_call(64, 32, 8, 128, 16, 256, 0, pa.PA_FP4_E2M1) == 2
    assert pa.pa_decode_kernels_per_call(1, 8, 1, 128, 16, 1, 0, pa.PA_FP4_E2M1) == 1  # a grid of one CTA
    assert pa.pa_decode_kernels_per_call(1, 8, 1, 128, 16, 1, 0, pa.PA_FP8_E4M3) == 2


def test_decode_of_nothing():
    c = Case(3, 8, 2, 128, 16, [0, 0, 0])
    assert not c.run().any() and not c.run(part=64).any() and not c.run(max_seq_len=100).any()
    assert status_word(c.ws) == 0


@pytest.mark.parametrize("part", [0, 32])
def test_decode_many_sequences(part):
    """More sequences than the 16-warp kernel's shared memory holds the lengths of."""
    lens = synth.uniform_ints(77, 2300, 0, 40).astype(np.int32)
    lens[1111] = 900
    c = Case(21, 8, 1, 128, 16, lens)
    c.check(c.run(part), seqs=[0, 1, 2, 1110, 1111, 1112, 2298, 2299] + list(range(100, 2300, 100)))
    assert status_word(c.ws) == 0


def test_decode_of_ranges_past_32_bits():
    """One sequence whose tiles, weighted as the ranges weigh them, number more than 2^31.  Its table repeats a few
    blocks; three tiles, the first and the last among them, hold keys whose scores are 200 above all others, so the
    output is the mean of their values (the other weights together are below 2^33 e^-200)."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    hkv, d, bs, n = 64, 64, 16, 8_400_004
    assert 4 * n * hkv > 1 << 31
    kp, vp = np.zeros((7, hkv, bs * 36), np.uint8), _random_pool(22, 7, hkv, bs, d)
    codes, scales = bs * d // 2, slice(bs * d // 2, None)
    kp[4:, :, :codes], kp[4:, :, scales] = 0x22, 0x38  # code 1 of scale 1: with q = 1 a score of 64 before its scale
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None] % 4
    where = [0, n // 2 + 1, n - 1]
    table[0, where] = torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda")
    q = torch.ones(1, hkv, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, float("nan"))
    ws = torch.zeros(pa.pa_decode_workspace_bytes(1, hkv, hkv, d), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([n * bs], dtype=torch.int32, device="cuda")
    pa.pa_decode_attention_fp4(out, q, to_torch(kp), to_torch(vp), 1.0, 0.5, table, lens, n * bs, 200.0 / 64.0, ws)
    v = kv4.values(vp[4:], d, bs).astype(np.float64) * 0.5  # [3][hkv][bs][d]
    want = v.transpose(1, 0, 2, 3).reshape(hkv, 3 * bs, d).mean(1)
    # weights equal up to the rounding of 2^x (2^-11 in f16 each), 48 sums in fp32, the output's rounding
    size = np.abs(v).transpose(1, 0, 2, 3).reshape(hkv, 3 * bs, d).mean(1)
    assert np.all(np.abs(widen(to_numpy(out))[0] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size)
    assert status_word(ws) == 0


def test_decode_one_long_sequence():
    c = Case(5, 8, 1, 128, 16, [20000])
    c.check(c.run())
    c.check(c.run(part=512))


@pytest.mark.parametrize("q_size", [1e-30, 1e30, 3e4])
def test_decode_takes_any_query_magnitude(q_size):
    c = Case(9, 8, 2, 128, 16, [70, 3, 200], q_size=q_size)
    c.check(c.run())


def test_decode_scores_far_apart_and_negative_scale():
    """One key far above the rest, equal keys, and a negative score scale."""
    c = Case(11, 4, 2, 64, 16, [90, 40], scales=(8.0, 0.5))  # scores of a few hundred
    c.check(c.run())
    c.scale = -c.scale
    c.check(c.run())
    c.kp[...] = 0  # every score 0: the mean
    c.check(c.run())


def test_decode_nan_reaches_only_its_heads():
    c = Case(12, 8, 2, 128, 16, [40, 50])
    blk = c.tables[1, 2]
    cut = c.bs * c.d // 2
    c.kp[blk, 1, cut + 3 * 8] = 0x7F  # a key of sequence 1, KV head 1
    got = widen(c.run())
    assert np.isnan(got[1, 4:]).all() and np.isfinite(got[0]).all() and np.isfinite(got[1, :4]).all()
    c.kp[blk, 1, cut + 3 * 8] = 0x30
    c.vp[blk, 0, cut + 3 * 8 + 5] = 0x7F  # a value group: dims 80..95 of KV head 0
    got = widen(c.run())
    nan = np.zeros((8, 128), bool)
    nan[:4, 80:96] = True
    assert np.array_equal(np.isnan(got[1]), nan) and np.isfinite(got[0]).all()


def test_decode_flags_bad_inputs():
    import paged_kv_cache_280_gb300 as pa

    c = Case(13, 8, 2, 128, 16, [40, 50])
    tables = c.tables.copy()
    tables[1, 1] = c.nb  # one past the pool: block 0 is read instead
    c.run(tables=tables)
    assert status_word(c.ws) == pa.PA_DEV_BAD_BLOCK_ID
    c.run(max_seq_len=45)
    assert status_word(c.ws) == pa.PA_DEV_BAD_SEQ_LEN
    with pytest.raises(pa.PAError) as e:
        import torch
        c.run(ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "PA_ERR_WORKSPACE_TOO_SMALL"


def test_decode_wait_timeout_is_reported():
    """A wait limit far below a DRAM round trip: the kernel reports it and the context stays usable.  The queries are
    in L2 and the pools, larger than it, are not, so that the first tiles are still on their way when they are wanted."""
    import paged_kv_cache_280_gb300 as pa

    c = Case(14, 32, 8, 128, 16, [8000] * 32)
    c.check(c.run(), seqs=[0])
    q, kp, vp, tab, lens = c.dev
    out = q.clone()
    try:
        pa.pa_debug_set_wait_limit_ns(1)
        pa.pa_decode_attention_fp4(out, q, kp, vp, *c.scales, tab, lens, 8000, c.scale, c.ws)
        assert status_word(c.ws) & pa.PA_DEV_WAIT_TIMEOUT
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    c.check(c.run(), seqs=[0, 31])


def test_decode_on_another_stream_and_captured():
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(15, 16, 4, 128, 16, [300, 17, 1000])
    want = c.run()
    assert np.array_equal(c.run(stream=torch.cuda.Stream()), want)
    q, kp, vp, tab, lens = c.dev
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_decode_attention_fp4(out, q, kp, vp, *c.scales, tab, lens, 1000, c.scale, c.ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert np.array_equal(to_numpy(out), want)


def test_one_workspace_for_decodes_over_both_pool_types():
    """The bf16 decode counts split pieces in its workspace and leaves the counts at zero; a 4-bit call between two of
    them, of another grid, must not disturb that."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(16, 8, 8, 128, 16, [700, 300, 90, 1200, 33])
    ws = torch.zeros(pa.pa_decode_workspace_bytes(5, 8, 8, 128), dtype=torch.uint8, device="cuda")
    pool = [to_torch(synth.normal(synth.stream_seed(17, i), c.nb * 8 * 16 * 128, "bf16").reshape(c.nb, 8, 16, 128)) for i in (1, 2)]
    q, tab, lens = to_torch(c.q), to_torch(c.tables), to_torch(c.lens)

    def bf16():
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_attention(out, q, *pool, tab, lens, 1200, c.scale, ws)
        return to_numpy(out)

    try:
        pa.pa_debug_set_merge_mode(1)
        first, fp4 = bf16(), c.run(ws=ws)
        assert np.array_equal(bf16(), first) and np.array_equal(c.run(ws=ws), fp4) and np.array_equal(bf16(), first)
    finally:
        pa.pa_debug_set_merge_mode(0)
    c.check(fp4)
    assert np.all(np.isfinite(widen(first)))


def test_copy_and_swap_of_4_bit_blocks():
    import torch
    import paged_kv_cache_280_gb300 as pa

    for d, bs, hkv in ((128, 16, 3), (64, 16, 1), (64, 32, 8), (128, 32, 2)):
        kp, vp = _random_pool(d, 9, hkv, bs, d), _random_pool(bs, 9, hkv, bs, d)
        dk, dv = to_torch(kp), to_torch(vp)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pairs = np.array([[1, 2], [7, 0]], np.int32)
        pa.pa_copy_blocks(dk, dv, to_torch(pairs), status=status)
        for p in (kp, vp):
            p[[2, 0]] = p[[1, 7]]
        assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp)
        stores = [torch.zeros((3, *kp.shape[1:]), dtype=torch.uint8).pin_memory() for _ in range(2)]
        ids = torch.tensor([8, 3, 5], dtype=torch.int32, device="cuda")
        pa.pa_swap_out(dk, dv, ids, *stores, status=status)
        torch.cuda.synchronize()
        assert np.array_equal(stores[0].numpy(), kp[[8, 3, 5]]) and np.array_equal(stores[1].numpy(), vp[[8, 3, 5]])
        dk[[8, 3, 5]], dv[[8, 3, 5]] = 0, 0
        pa.pa_swap_in(*stores, ids, dk, dv, status=status)
        assert np.array_equal(to_numpy(dk), kp) and np.array_equal(to_numpy(dv), vp) and status.item() == 0


def test_far_blocks_of_a_large_pool():
    """Offsets past 32 bits: the last blocks of a 4.7 GB pool, through append, unpacking and decode."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    nb, hkv, d, bs, n = 510_000, 8, 128, 16, 45
    kp, vp = (torch.zeros(nb, hkv, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2))
    assert kp.numel() > 1 << 32
    x = synth.normal(synth.stream_seed(21, 1), 2 * n * hkv * d, "bf16").reshape(2, n, hkv, d)
    blocks = np.array([nb - 1, nb - 3, 478_000], np.int32)
    slots = (blocks.astype(np.int64)[np.arange(n) // bs]) * bs + np.arange(n) % bs
    pa.pa_reshape_and_cache_fp4(to_torch(x[0]), to_torch(x[1]), kp, vp, to_torch(slots), 1.0, 1.0)
    host = [np.zeros((3, hkv, bs * 72), np.uint8) for _ in range(2)]
    kv4.append_fp4(x[0], x[1], *host, np.arange(n), bs, 1.0, 1.0)
    at = to_torch(blocks)
    for p, h in zip((kp, vp), host):
        assert np.array_equal(to_numpy(p[at.long()]), h)
    out = [torch.zeros(3, hkv, bs, d, device="cuda") for _ in range(2)]
    pa.pa_unpack_blocks_fp4(kp, vp, at, *out, 1.0, 1.0)
    assert np.array_equal(to_numpy(out[0]), kv4.values(host[0], d, bs).astype(np.float32))
    q = synth.normal(synth.stream_seed(21, 2), 8 * hkv * d, "bf16").reshape(1, 8 * hkv, d)
    o = torch.zeros(1, 8 * hkv, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(pa.pa_decode_workspace_bytes(1, 8 * hkv, hkv, d), dtype=torch.uint8, device="cuda")
    pa.pa_decode_attention_fp4(o, to_torch(q), kp, vp, 1.0, 1.0, at[None].contiguous(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"), n, 0.09, ws)
    ref, bound = kv4.decode_fp4(q, *host, 1.0, 1.0, np.array([[0, 1, 2]], np.int32), np.array([n]), 0.09, bs)
    assert np.all(np.abs(widen(to_numpy(o)) - ref) <= 2.0 ** -8 * (np.abs(ref) + bound) + bound)


@pytest.mark.parametrize("captured", [False, True])
def test_serving_steps_over_a_4_bit_cache(captured):
    """A prompt and decode steps as a server makes them: allocator, rotating append, the chunk's prefill over the
    unpacked blocks, then rotating append and decode per step, eager or captured in one graph."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    B, hq, hkv, d, bs, nb, steps = 3, 8, 2, 128, 16, 24, 3
    prompts = [37, 16, 61]
    table = kv4.cos_sin_table(128, d)
    dtable = to_torch(table)
    alloc = pa.Allocator(nb, bs, free_order=synth.permutation(3, nb).astype(np.int32))
    kp, vp = _random_pool(1, nb, hkv, bs, d), _random_pool(2, nb, hkv, bs, d)
    dkp, dvp = to_torch(kp), to_torch(vp)
    ks, vs, scale = 0.7, 0.3, float(1 / np.sqrt(d))

    def qkv(step, n):
        x = synth.normal(synth.stream_seed(50 + step, 1), n * (hq + 2 * hkv) * d, "bf16").reshape(n, hq + 2 * hkv, d)
        return x, (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])

    # the prompts, as one packed chunk
    slots = np.concatenate([(alloc.create(b), alloc.append(b, n)[0])[1] for b, n in enumerate(prompts)])
    pos = np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)
    x, (q, k, v) = qkv(0, sum(prompts))
    t = to_torch(x)
    q_rot = torch.empty(sum(prompts), hq, d, dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(q_rot, t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:], to_torch(pos), dtable, dkp, dvp, to_torch(slots),
                         k_scale=ks, v_scale=vs)
    tables, lens = alloc.export_tables(range(B), 8)
    ids = np.concatenate([tables[b, : -(-n // bs)] for b, n in enumerate(prompts)])
    scratch = [torch.zeros(len(ids), hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pa.pa_unpack_blocks_fp4(dkp, dvp, to_torch(ids), *scratch, ks, vs)
    at, dense = 0, np.zeros((B, 8), np.int32)
    for b, n in enumerate(prompts):
        m = -(-n // bs)
        dense[b, :m] = np.arange(at, at + m)
        at += m
    cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    out = torch.empty_like(q_rot)
    pa.pa_prefill_attention(out, q_rot, *scratch, to_torch(dense), to_torch(lens), to_torch(cu), max(prompts), scale)
    kv4.append_fp4(kv4.rotate_f32(k, pos, table, False), v, kp, vp, slots, bs, ks, vs)
    assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
    rq = kv4.to_bf16(kv4.rotate_f32(q, pos, table, False))
    assert np.array_equal(to_numpy(q_rot), rq)
    host = [kv4.to_bf16(kv4.values(p[ids], d, bs).astype(np.float32) * np.float32(s)) for p, s in ((kp, ks), (vp, vs))]
    for h, g in zip(host, scratch):
        live = np.zeros((len(ids), bs), bool)
        for b, n in enumerate(prompts):
            live[dense[b, np.arange(n) // bs], np.arange(n) % bs] = True
        assert np.array_equal(to_numpy(g).transpose(0, 2, 1, 3)[live], h.transpose(0, 2, 1, 3)[live])
    want = oracle.prefill_attention(rq, *host, dense, lens, cu, scale)
    assert np.all(np.abs(widen(to_numpy(out)) - want) <= 1e-2 + 1e-2 * np.abs(want))

    # decode steps
    buf = {"x": torch.empty(B, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda"),
           "pos": torch.empty(B, dtype=torch.int32, device="cuda"), "slots": torch.empty(B, dtype=torch.int64, device="cuda"),
           "tables": torch.empty(B, 8, dtype=torch.int32, device="cuda"), "lens": torch.empty(B, dtype=torch.int32, device="cuda")}
    q1 = torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda")
    o1 = torch.empty_like(q1)
    ws = torch.zeros(pa.pa_decode_workspace_bytes(B, hq, hkv, d), dtype=torch.uint8, device="cuda")

    def step():
        y = buf["x"]
        pa.pa_rope_and_cache(q1, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], buf["pos"], dtable, dkp, dvp, buf["slots"],
                             k_scale=ks, v_scale=vs)
        pa.pa_decode_attention_fp4(o1, q1, dkp, dvp, ks, vs, buf["tables"], buf["lens"], 8 * bs, scale, ws)

    graph = None
    for i in range(1, steps + 1):
        pos = alloc.export_tables(range(B), 8)[1].copy()
        slots, _ = alloc.append_batch(list(range(B)))
        tables, lens = alloc.export_tables(range(B), 8)
        x, (q, k, v) = qkv(i, B)
        for name, a in (("x", x), ("pos", pos), ("slots", slots), ("tables", tables), ("lens", lens)):
            buf[name].copy_(to_torch(a))
        if captured and i == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        kv4.append_fp4(kv4.rotate_f32(k, pos, table, False), v, kp, vp, slots, bs, ks, vs)
        assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
        rq = kv4.to_bf16(kv4.rotate_f32(q, pos, table, False))
        assert np.array_equal(to_numpy(q1), rq)
        ref, bound = kv4.decode_fp4(rq, kp, vp, ks, vs, tables, lens, scale, bs)
        assert np.all(np.abs(widen(to_numpy(o1)) - ref) <= 2.0 ** -8 * (np.abs(ref) + bound) + bound)
    assert status_word(ws) == 0


def test_a_captured_step_whose_inputs_come_from_two_streams():
    """The lengths and the rows are written in the graph, the rows on a second stream that joins before the append; the
    decode follows the append.  Each replay takes what the buffers then hold."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    hq, hkv, d, bs, nb, B = 8, 2, 128, 16, 12, 3
    gen = np.random.default_rng(5)
    steps = [kv4.to_bf16(gen.standard_normal((B, hq + 2 * hkv, d)).astype(np.float32)) for _ in range(3)]
    table = kv4.cos_sin_table(64, d)
    dtable, dsteps = to_torch(table), [to_torch(x) for x in steps]
    kp, vp = _random_pool(1, nb, hkv, bs, d), _random_pool(2, nb, hkv, bs, d)
    dkp, dvp = to_torch(kp), to_torch(vp)
    tables = np.arange(nb, dtype=np.int32).reshape(B, 4)[:, ::-1].copy()
    start = np.array([0, 15, 40], np.int32)
    dtables, lens = to_torch(tables), to_torch(start)
    given, x = (torch.empty_like(dsteps[0]) for _ in range(2))
    q_rot, out = (torch.empty(B, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.zeros(pa.pa_decode_workspace_bytes(B, hq, hkv, d), dtype=torch.uint8, device="cuda")
    rows = torch.arange(B, device="cuda")

    def step():
        main, side = torch.cuda.current_stream(), step.side
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.copy_(given)
        pos = lens.clone()
        at = pos.long()
        slots = dtables[rows, at // bs].long() * bs + at % bs
        lens.add_(1)
        main.wait_stream(side)
        pa.pa_rope_and_cache(q_rot, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, dtable, dkp, dvp, slots)
        pa.pa_decode_attention_fp4(out, q_rot, dkp, dvp, 1.0, 1.0, dtables, lens, 64, d ** -0.5, ws)

    step.side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, s in enumerate(steps):
        given.copy_(dsteps[i])
        graph.replay()
        pos = start + i
        slots = tables[np.arange(B), pos // bs].astype(np.int64) * bs + pos % bs
        k = kv4.rotate_f32(s[:, hq:hq + hkv], pos, table, False)
        kv4.append_fp4(k, s[:, hq + hkv:], kp, vp, slots, bs, 1.0, 1.0)
        rq = kv4.to_bf16(kv4.rotate_f32(s[:, :hq], pos, table, False))
        assert np.array_equal(to_numpy(dkp), kp) and np.array_equal(to_numpy(dvp), vp)
        assert np.array_equal(to_numpy(lens), pos + 1) and np.array_equal(to_numpy(q_rot), rq)
        ref, bound = kv4.decode_fp4(rq, kp, vp, 1.0, 1.0, tables, pos + 1, d ** -0.5, bs)
        assert np.all(np.abs(widen(to_numpy(out)) - ref) <= 2.0 ** -8 * (np.abs(ref) + bound) + bound)
    assert status_word(ws) == 0


def test_two_decodes_at_once():
    """Two streams, a workspace each: neither call's pieces reach the other's."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    cases = [Case(18, 32, 8, 128, 16, [2000, 31, 777, 4000]), Case(19, 8, 8, 64, 32, [3000, 1, 500])]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.zeros_like(c.dev[0]) for _ in range(8)] for c in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for c, s, o in zip(cases, streams, outs):
            q, kp, vp, tab, lens = c.dev
            pa.pa_decode_attention_fp4(o[i], q, kp, vp, *c.scales, tab, lens, int(c.lens.max()), c.scale, c.ws, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(np.array_equal(to_numpy(x), w) for x in o)


def test_two_graphs_of_one_workspace():
    """Calls of different grids captured with the same workspace and replayed in turn on one stream."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    cases = [Case(23, 8, 8, 128, 16, [40]), Case(24, 8, 8, 128, 32, [1500, 0, 700, 33])]
    want = [c.run() for c in cases]
    ws = torch.zeros(pa.pa_decode_workspace_bytes(4, 8, 8, 128), dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(c.dev[0]) for c in cases], []
    for c, o in zip(cases, outs):
        q, kp, vp, tab, lens = c.dev
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            pa.pa_decode_attention_fp4(o, q, kp, vp, *c.scales, tab, lens, int(c.lens.max()), c.scale, ws)
    for i in (0, 1, 0, 1, 1, 0):
        outs[i].fill_(7.0)
        graphs[i].replay()
        assert np.array_equal(to_numpy(outs[i]), want[i])
    assert status_word(ws) == 0
