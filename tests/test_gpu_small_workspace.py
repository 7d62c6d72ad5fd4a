"""GPU: a decode workspace that is too small to keep the merge counters of every grid apart from the partials."""
import numpy as np
import pytest

import synth
from gpu_cases import status_word, to_numpy, to_torch, widen

pytestmark = pytest.mark.gpu


def test_a_workspace_too_small_for_every_grids_counters():
    """A call that has no room for its partials behind the counters of the largest grid puts them where a larger grid's
    counters lie.  A later call of such a grid (of smaller heads, so that the same bytes suffice) must find them at zero."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def least(ctas, group, d):  # (the header gives the layout: a 256-byte head, a counter per CTA, two slots per CTA)
        slot = -(-group * (d + 2) // 4) * 16
        return 256 + -(-ctas * 4 // 256) * 256, slot, 256 + -(-ctas * 4 // 256) * 256 + 2 * ctas * slot

    behind = 256 + -(-sms * 8 * 4 // 256) * 256
    pools = {d: [to_torch(synth.normal(synth.stream_seed(41, i), 64 * 16 * d, "bf16").reshape(64, 1, 16, d)) for i in (1, 2)]
             for d in (64, 128)}

    def call(group, d, seqs, tiles, ws):
        q = to_torch(synth.normal(synth.stream_seed(42, group), seqs * group * d, "bf16").reshape(seqs, group, d))
        tab = to_torch((np.arange(seqs * tiles, dtype=np.int32) * 7 % 64).reshape(seqs, tiles))
        out = torch.full_like(q, float("nan"))
        pa.pa_decode_attention(out, q, *pools[d], tab, torch.full((seqs,), tiles * 16, dtype=torch.int32, device="cuda"),
                               tiles * 16, d ** -0.5, ws)
        return to_numpy(out)

    try:
        pa.pa_debug_set_merge_mode(1)
        most = {(g, d): pa.pa_decode_launch_info(4096, g, 1, d, 16, 8, pa.PA_BF16)[0] for g, d in ((1, 64), (3, 64), (2, 128))}
        best = None  # the pair of grids with the most counters under the first one's first written slot
        for g, d in ((3, 64), (2, 128)):
            for ga in range(2, most[g, d] + 1):
                start, slot, need = least(ga, g, d)
                for gb in range(ga // 8 * 8 + 8, most[1, 64] + 1, 8):
                    size = max(need, least(gb, 1, 64)[2])
                    if size < behind + 2 * ga * slot and (best is None or gb - (start + slot - 256) // 4 > best[0]):
                        best = gb - (start + slot - 256) // 4, g, d, ga, gb, size
        under, g, d, ga, gb, size = best
        assert under > 16
        want = call(1, 64, gb // 8, 8, torch.zeros(pa.pa_decode_workspace_bytes(gb // 8, 1, 1, 64), dtype=torch.uint8, device="cuda"))
        assert np.isfinite(widen(want)).all()
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        for _ in range(2):
            call(g, d, 1, ga, ws)
            assert np.array_equal(call(1, 64, gb // 8, 8, ws), want)
        assert status_word(ws) == 0
    finally:
        pa.pa_debug_set_merge_mode(0)
