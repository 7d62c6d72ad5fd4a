"""GPU: one decode workspace for calls whose grids differ."""
import numpy as np
import pytest

import synth
from gpu_cases import to_numpy, to_torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hq,hkv,d,bs", [("bf16", 8, 8, 128, 16), ("bf16", 32, 8, 128, 16), ("f32", 4, 4, 64, 32)])
def test_a_larger_grid_after_a_smaller_one(dtype, hq, hkv, d, bs):
    """With the merge in the decode kernel a call counts split pieces at its workspace's start, where the smaller call's
    partials must not have been."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    nb = 300
    pool = [to_torch(synth.normal(synth.stream_seed(31, i), nb * hkv * bs * d, dtype).reshape(nb, hkv, bs, d)) for i in (1, 2)]

    def call(n, tokens, ws):
        per = -(-tokens // bs)
        q = to_torch(synth.normal(synth.stream_seed(32, n), n * hq * d, dtype).reshape(n, hq, d))
        tab = (np.arange(n * per, dtype=np.int32) * 7 % nb).reshape(n, per)
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_attention(out, q, *pool, to_torch(tab), to_torch(np.full(n, tokens, np.int32)), tokens, d ** -0.5, ws)
        return to_numpy(out)

    def new():
        return torch.zeros(pa.pa_decode_workspace_bytes(3, hq, hkv, d), dtype=torch.uint8, device="cuda")

    try:
        pa.pa_debug_set_merge_mode(1)
        want, ws = call(3, 1200, new()), new()
        for _ in range(2):
            call(1, 100, ws)
            assert np.array_equal(call(3, 1200, ws), want)
    finally:
        pa.pa_debug_set_merge_mode(0)
