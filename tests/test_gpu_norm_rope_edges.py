"""GPU: the normed rotating append at the edges of what its call allows."""
import numpy as np
import pytest

from gpu_cases import to_torch
from oracle import kv4
from test_gpu_norm_rope import EPS
from test_gpu_rope import MAXP, _inputs

pytestmark = pytest.mark.gpu


def _call(q, k, v, w, pools, slots, pos, table, **kw):
    import torch
    import paged_kv_cache_280_gb300 as pa

    q_out, k_out = (torch.zeros(t.shape, dtype=t.dtype, device="cuda") for t in (q, k))
    pa.pa_norm_rope_and_cache(q_out, k_out, q, k, v, *w, EPS, pos, table, *pools, slots, **kw)
    return q_out, k_out


@pytest.mark.parametrize("dtype,pool", [("bf16", "fp4"), ("f32", "same")])
def test_norm_rope_inputs_and_pools_past_32_bits(dtype, pool):
    """Rows more than 2^32 elements apart, slots past 4 GiB of a pool: as from dense rows into a small pool."""
    import torch

    n, hq, hkv, d, bs = 3000, 6, 2, 128, 16
    _, dev = _inputs(41, n, hq, hkv, d, dtype, False)
    row = 1536000  # elements from one token to the next: the last one begins past 2^32
    if dtype == "f32":
        n, row = 1500, 2880000
        dev = [t[:n] for t in dev]
    total = (hq + 2 * hkv) * d
    big = torch.empty((n - 1) * row + total, dtype=dev[0].dtype, device="cuda")
    rows = big.as_strided((n, total), (row, 1))
    rows.copy_(torch.cat([t.flatten(1) for t in dev], 1))
    views, at = [], 0
    for t in dev:
        h = t.shape[1]
        views.append(rows[:, at:at + h * d].unflatten(1, (h, d)))
        at += h * d
    w = [torch.linspace(0.5, 2, d, device="cuda"), torch.linspace(-1, 1.5, d, device="cuda")]
    pos, table = to_torch((np.arange(n) % MAXP).astype(np.int32)), to_torch(kv4.cos_sin_table(MAXP, d))
    blocks = -(-n // bs)
    shape = (bs * 72,) if pool == "fp4" else (bs, d)
    rec = hkv * int(np.prod(shape)) * (1 if pool == "fp4" else 4)
    shift = (1 << 32) // rec + 5
    small, large = ([torch.zeros((nb, hkv, *shape), dtype=torch.uint8 if pool == "fp4" else dev[0].dtype, device="cuda") for _ in range(2)]
                    for nb in (blocks, blocks + shift))
    slots = torch.arange(n, device="cuda")
    want = _call(*dev, w, small, slots, pos, table)
    got = _call(*views, w, large, slots + shift * bs, pos, table)
    for a, b in zip(want + tuple(small), got + tuple(p[shift:] for p in large)):
        assert torch.equal(a, b)
    assert not large[0][:shift].any() and not large[1][:shift].any()


@pytest.mark.parametrize("d", [64, 128])
def test_norm_rope_weights_aligned_to_4_bytes(d):
    import torch

    n, hq, hkv, bs = 70, 5, 3, 32
    _, dev = _inputs(42, n, hq, hkv, d, "bf16", True)
    w = [torch.linspace(0.5, 2, d, device="cuda"), torch.linspace(-1, 1.5, d, device="cuda")]
    odd = []
    for t in w:
        x = torch.empty(d + 1, device="cuda")[1:]
        x.copy_(t)
        assert x.data_ptr() % 8 == 4
        odd.append(x)
    pos, table, slots = to_torch(np.arange(n, dtype=np.int32)), to_torch(kv4.cos_sin_table(MAXP, d)), torch.arange(n, device="cuda")
    new = lambda: [torch.zeros(3, hkv, bs, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]  # noqa: E731
    a, b = new(), new()
    for x, y in zip(_call(*dev, w, a, slots, pos, table) + tuple(a), _call(*dev, odd, b, slots, pos, table) + tuple(b)):
        assert torch.equal(x, y)


def test_norm_rope_captured_twice_and_replayed_at_once():
    """Two captured appends into different slots of one pool, on two streams: what they give one after the other."""
    import torch

    n, hq, hkv, d, bs = 300, 8, 2, 128, 16
    _, dev = _inputs(43, 2 * n, hq, hkv, d, "bf16", True)
    halves = [[t[i * n:(i + 1) * n] for t in dev] for i in range(2)]
    w = [torch.linspace(0.5, 2, d, device="cuda")] * 2
    pos, table = to_torch((np.arange(n) % MAXP).astype(np.int32)), to_torch(kv4.cos_sin_table(MAXP, d))
    slots = [torch.arange(n, device="cuda") * 2 + i for i in range(2)]  # neighbours in every block
    new = lambda: [torch.zeros(-(-2 * n // bs), hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in range(2)]  # noqa: E731
    want = new()
    rows = [_call(*h, w, want, s, pos, table, k_scale=0.02, v_scale=0.02) for h, s in zip(halves, slots)]
    pools, outs, graphs, streams = new(), [], [], [torch.cuda.Stream() for _ in range(2)]
    for h, s, st in zip(halves, slots, streams):
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(_call(*h, w, pools, s, pos, table, k_scale=0.02, v_scale=0.02))
        graphs.append(g)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want + [t for r in rows for t in r], pools + [t for r in outs for t in r]):
        assert torch.equal(a, b)
