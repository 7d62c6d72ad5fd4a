"""GPU: a conversation over a quantised cache, step by step as a serving loop makes it: normed rotating append of a prompt,
prompt attention over its own keys, then a second turn's append and chunk attention over the cache, then a decode.

Every stage is compared with float64 from the inputs that the stage was given (its predecessor's outputs included).
"""
import numpy as np
import pytest

from gpu_cases import to_numpy, to_torch, widen
from oracle import chunks, kv4

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.mark.parametrize("kind,d", [("fp8", 128), ("fp4", 128), ("fp4", 64)])
def test_conversation(kind, d):
    import torch
    import paged_kv_cache_280_gb300 as pa

    hq, hkv, bs, ks, vs, scale = 8, 2, 16, 0.02, 0.03, d ** -0.5
    prompts, turns = [37, 150, 1], [5, 140, 33]
    rng = np.random.default_rng(d)
    lib = pa.Allocator(64, bs, free_order=rng.permutation(64).astype(np.int32))
    shape = (64, hkv, bs, d) if kind == "fp8" else (64, hkv, pa.fp4_block_bytes(d, bs))
    kp, vp = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.from_numpy(kv4.cos_sin_table(512, d)).cuda()
    qw, kw = (torch.from_numpy(rng.uniform(0.5, 2, d).astype(np.float32)).cuda() for _ in range(2))
    ws = torch.zeros(pa.pa_prefill_workspace_bytes(max(turns), hq, hkv, d), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for s in range(3):
        lib.create(s)

    def project(lens, first):
        """(normed, turned q; turned k; v; starts) of new tokens, which are appended."""
        total = sum(lens)
        x = torch.from_numpy(rng.standard_normal((total, hq + 2 * hkv, d)).astype(np.float32)).to(torch.bfloat16).cuda()
        slots = np.concatenate([lib.append(s, n)[0] for s, n in enumerate(lens)])
        pos = np.concatenate([np.arange(f, f + n) for f, n in zip(first, lens)]).astype(np.int32)
        q, k, v = torch.empty_like(x[:, :hq].contiguous()), torch.empty_like(x[:, hq:hq + hkv].contiguous()), x[:, hq + hkv:]
        pa.pa_norm_rope_and_cache(q, k, x[:, :hq], x[:, hq:hq + hkv], v, qw, kw, EPS, to_torch(pos), table, kp, vp,
                                  to_torch(slots), k_scale=ks, v_scale=vs, status=status)
        for got, part, w in ((q, x[:, :hq], qw), (k, x[:, hq:hq + hkv], kw)):
            want = kv4._rotate(chunks.head_norm(to_numpy(part), w.cpu().numpy(), EPS), pos, table.cpu().numpy().astype(np.float64), False)
            # fp32 to 2^-15 of the row's largest, then one rounding
            slack = 2.0 ** -15 * np.abs(want).max(-1, keepdims=True)
            assert np.all(np.abs(widen(to_numpy(got)) - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack))
        return q, k, v, np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)

    def near(got, want, bound):
        assert np.all(np.abs(widen(to_numpy(got)) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound))

    q, k, v, starts = project(prompts, [0] * 3)
    out = torch.empty_like(q)
    pa.pa_prompt_attention(out, q, k, v, to_torch(starts), max(prompts), scale, status=status)
    near(out, *chunks.prompts(to_numpy(q), to_numpy(k), to_numpy(v), starts, scale))

    attend = pa.pa_prefill_attention_fp8 if kind == "fp8" else pa.pa_prefill_attention_fp4
    for news in (turns, [1, 1, 1]):
        q, k, v, starts = project(news, [lib.length(s) for s in range(3)])
        most = max(len(lib.table(s)) for s in range(3))
        tables, lens = lib.export_tables(range(3), most)
        out = torch.empty_like(q)
        attend(out, q, kp, vp, ks, vs, to_torch(tables), to_torch(lens), to_torch(starts), max(news), scale, ws)
        near(out, *chunks.chunks(to_numpy(q), to_numpy(kp), to_numpy(vp), kind, ks, vs, tables, lens, starts, scale, bs))
    decode = pa.pa_decode_attention_fp8 if kind == "fp8" else pa.pa_decode_attention_fp4
    dws = torch.zeros(pa.pa_decode_workspace_bytes(3, hq, hkv, d), dtype=torch.uint8, device="cuda")
    one = torch.empty_like(out)
    decode(one, q, kp, vp, ks, vs, to_torch(tables), to_torch(lens), int(lens.max()), scale, dws)
    want, bound = chunks.chunks(to_numpy(q), to_numpy(kp), to_numpy(vp), kind, ks, vs, tables, lens, starts, scale, bs)
    near(one, want, 2.2 * bound)  # the decode divides by the rounded weights' sum: twice their rounding
    assert status.item() == 0 and int(ws[:4].view(torch.int32).item()) == 0
