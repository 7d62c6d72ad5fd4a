"""The checks of the normed rotating append, the prompt attention and the chunk attention over quantised pools: bad calls come
back from the host (no GPU needed)."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_280_gb300 as pa

FAKE = ctypes.c_void_p(1 << 20)  # 16-byte aligned, never dereferenced
OTHER = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 8)
TWO = ctypes.c_void_p((1 << 20) + 2)
INVALID, UNSUPPORTED = 1, 2
NAN, INF = float("nan"), float("inf")


def _norm(**kw):
    a = dict(q_out=OTHER, k_out=None, q=FAKE, qs=8 * 128, k=FAKE, ks=2 * 128, v=FAKE, vs=2 * 128, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE,
             table=FAKE, maxp=100, rot=128, inter=0, kp=FAKE, vp=FAKE, slots=FAKE, n=4, hq=8, hkv=2, d=128, bs=16, nb=10,
             dt=pa.PA_BF16, pdt=pa.PA_BF16, ksc=1.0, vsc=1.0, status=None, stream=None)
    a.update(kw)
    return pa._lib.pa_norm_rope_and_cache(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), 0), (dict(n=0, q=None, k=None, kw=None), 0), (dict(n=-1), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(kw=None), INVALID), (dict(qw=None), INVALID),
    (dict(kw=TWO), INVALID), (dict(qw=TWO), INVALID), (dict(k_out=ODD), INVALID), (dict(k_out=FAKE, ks=4 * 128), INVALID),
    (dict(rot=144), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=48, pdt=pa.PA_FP4_E2M1), UNSUPPORTED),
    (dict(dt=pa.PA_FP8_E4M3), UNSUPPORTED), (dict(pdt=pa.PA_F32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(ksc=0.0), INVALID), (dict(vsc=NAN), INVALID), (dict(qs=8 * 128 - 8), INVALID), (dict(vs=-256), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(vp=ODD), INVALID), (dict(q_out=FAKE, qs=12 * 128), INVALID),
    (dict(n=1 << 29), UNSUPPORTED),
])
def test_norm_rope_refusals(kw, want):
    assert _norm(**kw) == want


def _prompt(**kw):
    a = dict(out=OTHER, q=FAKE, qs=8 * 128, k=FAKE, ks=2 * 128, v=FAKE, vs=2 * 128, cu=FAKE, b=2, t=10, most=8, hq=8, hkv=2, d=128,
             scale=0.1, dt=pa.PA_BF16, status=None, stream=None)
    a.update(kw)
    return pa._lib.pa_prompt_attention(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(t=0), 0), (dict(most=0), 0), (dict(t=0, q=None), 0), (dict(t=-1), INVALID), (dict(most=-1), INVALID), (dict(b=0), INVALID),
    (dict(dt=pa.PA_F32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(hq=7), INVALID), (dict(hq=18, qs=18 * 128), UNSUPPORTED),
    (dict(hkv=0), INVALID), (dict(b=65536), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID),
    (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(qs=8 * 128 - 8), INVALID), (dict(ks=2 * 128 + 4), INVALID),
    (dict(vs=0), INVALID), (dict(vs=1 << 40), UNSUPPORTED), (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(k=ODD), INVALID),
    (dict(v=ODD), INVALID), (dict(out=ODD), INVALID), (dict(cu=None), INVALID), (dict(cu=TWO), INVALID), (dict(status=TWO), INVALID),
])
def test_prompt_refusals(kw, want):
    assert _prompt(**kw) == want


def _chunk(call, **kw):
    a = dict(out=OTHER, q=FAKE, kp=FAKE, vp=FAKE, ks=1.0, vs=1.0, tables=FAKE, mb=4, lens=FAKE, cu=FAKE, b=2, t=10, most=8, hq=8, hkv=2,
             d=128, bs=16, nb=10, scale=0.1, ws=FAKE, wsb=1 << 30, stream=None)
    a.update(kw)
    return call(*a.values())


@pytest.mark.parametrize("call", [pa._lib.pa_prefill_attention_fp8, pa._lib.pa_prefill_attention_fp4])
@pytest.mark.parametrize("kw,want", [
    (dict(t=0), 0), (dict(most=0), 0), (dict(t=-1), INVALID), (dict(most=-1), INVALID), (dict(b=0), INVALID), (dict(mb=0), INVALID),
    (dict(nb=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(hq=7), INVALID), (dict(hq=18), UNSUPPORTED),
    (dict(b=65536), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=NAN), INVALID), (dict(ks=0.0), INVALID), (dict(vs=INF), INVALID),
    (dict(vs=-1.0), INVALID), (dict(ks=1e-38, scale=1e-30), INVALID), (dict(ks=1e38, scale=1e30), INVALID), (dict(out=None), INVALID),
    (dict(q=ODD), INVALID), (dict(kp=None), INVALID), (dict(vp=ODD), INVALID), (dict(tables=None), INVALID), (dict(tables=TWO), INVALID),
    (dict(lens=None), INVALID), (dict(cu=TWO), INVALID), (dict(ws=None), INVALID), (dict(ws=ODD), INVALID),
])
def test_chunk_refusals(call, kw, want):
    assert _chunk(call, **kw) == want


def test_fp8_chunks_need_head_dim_128():
    assert _chunk(pa._lib.pa_prefill_attention_fp8, d=64) == UNSUPPORTED


def test_workspace_size_refusals():
    n = ctypes.c_size_t(0)
    call = pa._lib.pa_prefill_workspace_bytes
    assert call(4, 8, 2, 128, None) == INVALID and call(-1, 8, 2, 128, ctypes.byref(n)) == INVALID
    assert call(4, 7, 2, 128, ctypes.byref(n)) == INVALID and call(4, 8, 0, 128, ctypes.byref(n)) == INVALID


def test_binding_refusals():
    """What the C side cannot see: CPU tensors, wrong types and shapes, heads that are not contiguous."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 128)
    ids = torch.zeros(3, dtype=torch.int32)
    pool4 = torch.zeros(5, 2, pa.fp4_block_bytes(128, 16), dtype=torch.uint8)
    pool8 = torch.zeros(5, 2, 16, 128, dtype=torch.uint8)
    with pytest.raises(pa.PAError, match="go together"):
        pa.pa_norm_rope_and_cache(k, None, k, k, k, None, k[0, 0], 1e-6, ids, k[0], pool4, pool4, ids)
    with pytest.raises(ValueError, match="k must be a CUDA"):
        pa.pa_norm_rope_and_cache(None, None, None, k, k, None, k[0, 0], 1e-6, ids, k[0], pool4, pool4, ids)
    with pytest.raises(pa.PAError, match="whole rows"):
        pa.pa_norm_rope_and_cache(None, None, None, k, k, None, k[0, 0], 1e-6, ids, k[0], pool4[..., :100], pool4, ids)
    with pytest.raises(ValueError, match="out must be a CUDA"):
        pa.pa_prompt_attention(k, k, k, k, ids, 3, 0.1)
    with pytest.raises(ValueError, match="out must be a CUDA"):
        pa.pa_prefill_attention_fp8(k, k, pool8, pool8, 1.0, 1.0, ids[None], ids[:1], ids[:2], 3, 0.1, pool4)
    with pytest.raises(pa.PAError, match="pool"):
        pa.pa_prefill_attention_fp8(k, k, pool8.float(), pool8, 1.0, 1.0, ids[None], ids[:1], ids[:2], 3, 0.1, pool4)
    with pytest.raises(pa.PAError, match="pool"):
        pa.pa_prefill_attention_fp8(k[..., :64], k[..., :64], pool8, pool8, 1.0, 1.0, ids[None], ids[:1], ids[:2], 3, 0.1, pool4)
    with pytest.raises(pa.PAError, match="uint8"):
        pa.pa_prefill_attention_fp4(k, k, pool8, pool8, 1.0, 1.0, ids[None], ids[:1], ids[:2], 3, 0.1, pool4)


def test_oracle_pins():
    """The oracle itself: two keys by hand, and its sequence and head bookkeeping against a direct double loop."""
    from oracle import chunks, kv4

    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    k = np.array([[[0.0, 1.0]], [[np.log(3.0), 0.0]]])
    v = np.array([[[4.0, -8.0]], [[8.0, 0.0]]])
    out, _ = chunks.causal(q, k, v, 0, 1.0, 0.0)
    assert np.allclose(out[0, 0], [4, -8]) and np.allclose(out[1, 0], (np.exp(2) * v[0, 0] + v[1, 0]) / (np.exp(2) + 1))
    out, _ = chunks.causal(q[:1], k, v, 1, 1.0, 0.0)
    assert np.allclose(out[0, 0], [7, -2])
    rng = np.random.default_rng(1)
    q, k, v = (kv4.to_bf16(rng.standard_normal((9, h, 64)).astype(np.float32)) for h in (4, 2, 2))
    out, _ = chunks.prompts(q, k, v, [1, 4, 4, 8], 0.3)
    assert np.isnan(out[[0, 8]]).all()
    w = [kv4.widen32(x).astype(np.float64) for x in (q, k, v)]
    for i, first in ((2, 1), (3, 1), (7, 4)):
        for h in range(4):
            p = np.exp(np.array([w[0][i, h] @ w[1][j, h // 2] for j in range(first, i + 1)]) * 0.3)
            assert np.allclose(out[i, h], (p / p.sum()) @ w[2][first:i + 1, h // 2])
    y = chunks.head_norm(np.array([[[3.0, 4.0]]], np.float32), np.array([1.0, 2.0], np.float32), 0.0)
    assert np.allclose(y, [[[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]]])
