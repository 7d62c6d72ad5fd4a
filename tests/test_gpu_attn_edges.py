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
