"""GPU: prompt attention and chunk attention over quantised pools at the edges of what their calls allow, against the definition
in float64."""
import numpy as np
import pytest

from oracle import chunks
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
