"""GPU: prompt attention and chunk attention over quantised pools at the edges of what their calls allow, against the definition
in float64."""
import numpy as np
import pytest

from gpu_cases import to_numpy, to_torch, widen
from oracle import chunks, kv4
from test_gpu_prefill_quant import KINDS, Case
from test_gpu_prompt import _check, _inputs, _run

pytestmark = pytest.mark.gpu


def test_prompts_of_offsets_past_32_bits_are_flagged():
    """A start below 0 and an end whose difference leaves 32 bits; the sequences around it are computed."""
    import paged_kv_cache_280_gb300 as pa

    host, dev = _inputs(21, 40, 4, 2, 64, False)
    for a, b in ((-5, 2 ** 31 - 1), (-(2 ** 31), 2 ** 31 - 1), (-(2 ** 31), 12)):
        got, status = _run(*dev, np.array([0, 12, a, b, 12, 40]), 0.1, max_len=1 << 30)
        assert status == pa.PA_DEV_BAD_SEQ_LEN
        _check(got, *chunks.prompts(*host, [0, 12, 12, 40], 0.1))


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_of_offsets_past_32_bits_are_flagged(kind, d):
    import paged_kv_cache_280_gb300 as pa

    c = Case(822, kind, [40, 30, 300, 30, 200], [12, 0, 0, 0, 28], 4, 2, d, 16)
    want, bound = c.want()
    for a, b in ((-5, 2 ** 31 - 1), (-(2 ** 31), 2 ** 31 - 1), (-(2 ** 31), 12)):
        c.starts = np.array([0, 12, a, b, 12, 40], np.int32)
        c.device()
        got = c.run()
        assert c.status() == pa.PA_DEV_BAD_SEQ_LEN
        _check(got, want, bound)


def test_tens_of_thousands_of_prompts_and_a_bound_of_all_tokens():
    """As many prompts as a call takes, nearly all of one token (whose output is its value, exactly), a bound on the lengths that
    only the sum of them keeps, and longer prompts at the ends and between."""
    import torch

    hq, hkv, d, n = 64, 8, 64, 65535
    lens = np.ones(n, np.int64)
    lens[[0, 31000, n - 1]] = 150, 61, 200
    lens[[5, 6, 40000]] = 0
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    total = int(starts[-1])
    x = torch.randn(total, hq + 2 * hkv, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    got, status = _run(q, k, v, starts, 0.125, max_len=1 << 30)
    assert status == 0
    single = torch.tensor(np.repeat(lens == 1, lens), device="cuda")
    assert torch.equal(got[single], v[single].repeat_interleave(hq // hkv, 1))
    for b in (0, 31000, n - 1):
        rows = slice(int(starts[b]), int(starts[b + 1]))
        host = [t[rows].contiguous().view(torch.int16).cpu().numpy().view(np.uint16) for t in (q, k, v)]
        _check(got[rows], *chunks.prompts(*host, [0, int(lens[b])], 0.125))


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("lens,news,hq,hkv", [([300, 140], [60, 140], 4, 2), ([5001, 77], [5, 77], 8, 1)])
@pytest.mark.parametrize("scale", [2e-8, 2e-25, 2e-36])
def test_chunks_zero_rows_under_the_smallest_scales(kind, d, lens, news, hq, hkv, scale):
    """A row of zeros weighs all the keys that it sees the same, whatever the scales, in units that are cut and that are not."""
    c = Case(830 + d, kind, lens, news, hq, hkv, d, 16, scale=scale)
    c.q[[0, 3, len(c.q) - 1]] = 0
    c.q[2, 1] = 0
    c.q[4, 0] = 0x8000  # negative zeros
    c.check(c.run())
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("scale", [1.0, 8.0, 1e30])
def test_chunks_largest_rows_over_keys_of_zeros(kind, d, scale):
    """Query rows at bf16's end, whose factor times the scale leaves fp32: scores of 0 all the same."""
    c = Case(840 + d, kind, [300, 140], [60, 140], 4, 2, d, 16, size=5e37, scale=scale)
    if kind == "fp8":
        c.kp[c.kp != 0x7F] &= 0x80
    else:
        c.kp[:, :, : 16 * d // 2] &= 0x88
    c.check(c.run())
    assert c.status() == 0


def _near(got, want, v_top, weight_eps, where=""):
    """Where the scores are exact: weights rounded (relative weight_eps) in the product with V, their exponents' fp32 rounding and
    the sums' (2^-16 together), and the output's."""
    g = widen(to_numpy(got))
    assert np.all(np.isfinite(g)), where
    err, limit = np.abs(g - want), (weight_eps + 2.0 ** -16) * v_top * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert np.all(err <= limit), f"{where}: max |err| {err.max():.3e}, {np.max(err / limit):.2f} of the bound"


def _one_element_rows(shape, size, seed):
    """Query rows with one element that is not 0, +-size: their products with keys are exact in fp32, whatever the size."""
    rng = np.random.default_rng(seed)
    q = np.zeros(shape, np.float32)
    at = rng.integers(0, shape[2], shape[:2])
    np.put_along_axis(q, at[..., None], rng.choice([-size, size], shape[:2])[..., None], 2)
    return kv4.to_bf16(q)


LARGE = [(2.0 ** 10, 1.0), (2.0 ** 17, 1.0), (2.0 ** 26, 1.0), (2.0 ** 33, 2.0), (2.0 ** 70, 1.0), (2.0 ** 124, 1.0), (2.0 ** 124, 2.0 ** 20),
         (1.0, 2.0 ** 40), (2.0 ** 100, 2.0 ** 100)]


@pytest.mark.parametrize("size,scale", LARGE)
@pytest.mark.parametrize("hq,hkv,d,lens", [(8, 2, 128, [300, 1, 700]), (4, 4, 64, [129, 520])])
def test_prompts_of_exact_scores_however_large(hq, hkv, d, lens, size, scale):
    """Scores past every power of two that fp32 and the weights have: the largest take all, in equal parts where they are equal."""
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, k, v), (_, dk, dv) = _inputs(31 + d, int(starts[-1]), hq, hkv, d, False)
    k = kv4.to_bf16(np.round(widen(k) * 2) / 2)  # few values, so that many keys share the largest score
    q = _one_element_rows(q.shape, size, 5)
    got, status = _run(to_torch(q), to_torch(k), dv, starts, scale)
    assert status == 0
    _near(got, chunks.prompts(q, k, v, starts, np.float64(scale))[0], np.abs(widen(v)).max(), chunks.EPS_BF16)


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("size,scale", LARGE)
@pytest.mark.parametrize("lens,news,hq,hkv", [([300, 140], [60, 140], 4, 2), ([5001, 77, 900], [5, 77, 200], 8, 1)])
def test_chunks_of_exact_scores_however_large(kind, d, lens, news, hq, hkv, size, scale):
    """The same over pools, in whole and in cut units, of one tile and of two."""
    c = Case(850 + d, kind, lens, news, hq, hkv, d, 16, scale=scale)
    c.q = _one_element_rows(c.q.shape, size, 6)
    got = c.run()
    assert c.status() == 0
    top = np.nanmax(np.abs(chunks.pool_values(c.vp, kind, d, 16))) * c.vs
    _near(got, c.want()[0], top, chunks.EPS_F16)


@pytest.mark.parametrize("common", [2.0 ** 12, 2.0 ** 16, 2.0 ** 19])
def test_prompts_of_large_scores_that_differ_little(common):
    """scale q k is a large number that all keys share plus one of 0 .. 4: only the small one counts."""
    starts = np.array([0, 700, 1000], np.int32)
    (q, k, v), (_, _, dv) = _inputs(33, 1000, 4, 2, 128, False)
    q, k = np.zeros(q.shape, np.float32), np.zeros(k.shape, np.float32)
    q[..., 0], q[..., 1] = common, 1
    k[..., 0], k[..., 1] = 1, np.random.default_rng(7).integers(0, 5, k.shape[:2])
    q, k = kv4.to_bf16(q), kv4.to_bf16(k)
    got, status = _run(to_torch(q), to_torch(k), dv, starts, 1.0)
    assert status == 0
    _near(got, chunks.prompts(q, k, v, starts, 1.0)[0], np.abs(widen(v)).max(), chunks.EPS_BF16)


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_leave_rows_behind_the_last_sequence(kind, d):
    """Rows of the batch past the last chunk are left as they were, and what their queries hold reaches nothing."""
    c = Case(860 + d, kind, [300, 90, 1500], [130, 1, 40], 6, 2, d, 16)
    want, bound = c.want()
    n = len(c.q)
    c.q = np.concatenate([c.q, np.full((9, *c.q.shape[1:]), 0x7FC0, np.uint16)])  # NaN
    got = c.run()
    assert c.status() == 0 and (got[n:] == 7).all()
    _check(got[:n], want, bound)


@pytest.mark.parametrize("kind,d", [("fp8", 128), ("fp4", 64)])
def test_chunks_of_as_many_sequences_as_a_call_takes(kind, d):
    """65535 sequences, over a hundred blocks that they share: most of one token, whose output is its value; some with no new token,
    some longer, at the ends and between."""
    import torch

    b, hq, hkv, bs, shared = 65535, 8, 2, 16, 100
    c = Case(870 + d, kind, [16] * shared, [1] * shared, hq, hkv, d, bs, poison=False)
    rng = np.random.default_rng(8)
    c.lens, c.news = np.ones(b, np.int32), np.ones(b, np.int32)
    longer = [0, 1, 40000, b - 1]
    c.lens[longer], c.news[longer] = [300, 40, 513, 77], [20, 1, 130, 33]
    c.news[[2, 3, 50000, b - 2]] = 0
    c.starts = np.concatenate([[0], np.cumsum(c.news)]).astype(np.int32)
    c.tables = rng.integers(0, shared, (b, 33)).astype(np.int32)
    c.q = kv4.to_bf16(rng.standard_normal((int(c.starts[-1]), hq, d)).astype(np.float32))
    got = c.run()
    assert c.status() == 0
    want, bound = c.want(longer)
    for s in longer:
        rows = slice(int(c.starts[s]), int(c.starts[s + 1]))
        _check(got[rows], want[rows], bound[rows])
    single = np.flatnonzero((c.lens == 1) & (c.news == 1))
    v = chunks.pool_values(c.vp, kind, d, bs)[c.tables[single, 0], :, 0] * np.float64(np.float32(c.vs))
    rows = torch.as_tensor(c.starts[single], dtype=torch.int64, device="cuda")
    _near(got[rows], np.repeat(v, hq // hkv, 1), np.abs(v).max(), 0.0)
