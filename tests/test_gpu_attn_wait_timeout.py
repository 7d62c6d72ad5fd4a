"""GPU: a wait of the prompt and chunk attention that runs out is reported, and the context stays usable.

Every wait of the pipeline's roles is bounded.  Some last as long as a piece of the work (the next query rows' place, the entries of
the pieces to come); with the limit cut to a nanosecond (pa_debug_set_wait_limit_ns) those run out on long contexts: the call comes
back with PA_DEV_WAIT_TIMEOUT in its status word, its roles having waited for their own copies and matrix products.  With the limit
restored, the same call on the same buffers gives what it gave before.  No GPU fault is provoked: the waits have a short limit."""
import numpy as np
import pytest

from test_gpu_prefill_quant import KINDS, Case
from test_gpu_prompt import _inputs, _run

pytestmark = pytest.mark.gpu


def _with_short_limit(call):
    import torch
    import paged_kv_cache_280_gb300 as pa

    try:
        pa.pa_debug_set_wait_limit_ns(1)
        status = call()
        torch.cuda.synchronize()
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    return status() if callable(status) else status


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_whose_waits_run_out(d):
    import torch
    import paged_kv_cache_280_gb300 as pa

    starts = np.array([0, 65536], np.int32)
    _, dev = _inputs(51, 65536, 2, 1, d, False)
    want, status = _run(*dev, starts, d ** -0.5)
    assert status == 0
    status = _with_short_limit(lambda: _run(*dev, starts, d ** -0.5)[1])
    assert status == pa.PA_DEV_WAIT_TIMEOUT, f"status {status:#x}"
    again, status = _run(*dev, starts, d ** -0.5)
    assert status == 0 and torch.equal(again, want)


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_whose_waits_run_out(kind, d):
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(52, kind, [131072], [5], 8, 1, d, 32, poison=False)
    b = 200  # sequences that share their blocks
    c.tables, c.lens, c.news = np.repeat(c.tables, b, 0), np.repeat(c.lens, b), np.repeat(c.news, b)
    c.starts = (5 * np.arange(b + 1)).astype(np.int32)
    c.q = np.tile(c.q, (b, 1, 1))
    c.device()
    want = c.run().clone()
    assert c.status() == 0

    def call():
        c.run()
        return c.status

    status = _with_short_limit(call)
    assert status == pa.PA_DEV_WAIT_TIMEOUT, f"status {status:#x}"
    assert torch.equal(c.run(), want) and c.status() == 0
