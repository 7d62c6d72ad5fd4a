"""GPU: attention over packed prompts (pa_prompt_attention) against the definition in float64."""
import numpy as np
import pytest

import synth
from gpu_cases import to_numpy, to_torch, widen
from oracle import chunks

pytestmark = pytest.mark.gpu


def _inputs(seed, total, hq, hkv, d, fused, size=1.0):
    x = synth.normal(synth.stream_seed(seed, 1), max(1, total) * (hq + 2 * hkv) * d, "f32").reshape(-1, hq + 2 * hkv, d)[:total]
    x[:, :hq] *= size
    x = (np.ascontiguousarray(x).view(np.uint32) >> 16).astype(np.uint16)  # bf16 bits
    host = (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:])
    if fused:
        t = to_torch(x)
        return host, (t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:])
    return host, tuple(to_torch(np.ascontiguousarray(a)) for a in host)


def _check(got, want, bound, rows=None):
    g = widen(to_numpy(got))
    if rows is not None:
        g, want, bound = g[rows], want[rows], bound[rows]
    assert np.all(np.isfinite(g))
    err, limit = np.abs(g - want), bound + 2.0 ** -8 * (np.abs(want) + bound)
    assert np.all(err <= limit), f"max |err| {err.max():.3e}, {np.max(err / limit):.2f} of the bound at {np.unravel_index(np.argmax(err / limit), err.shape)}"


def _run(q, k, v, starts, scale, max_len=None, before=7.0, **kw):
    import torch
    import paged_kv_cache_280_gb300 as pa

    out = torch.full(q.shape, before, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    most = int(np.diff(starts).max()) if max_len is None else max_len
    pa.pa_prompt_attention(out, q, k, v, to_torch(np.asarray(starts, np.int32)), most, scale, status=status, **kw)
    return out, int(status.item())


@pytest.mark.parametrize("hq,hkv,d,fused", [(1, 1, 64, False), (4, 4, 128, True), (8, 4, 64, True), (6, 2, 128, False), (8, 2, 128, True),
                                            (10, 2, 64, False), (6, 1, 128, True), (14, 2, 128, True), (16, 2, 64, False), (8, 1, 128, True)])
def test_prompts_ragged(hq, hkv, d, fused):
    """Lengths around the tiles' and stages' borders, empty sequences, rows of no sequence on both sides."""
    lens = [1, 0, 2, 31, 32, 33, 64, 127, 128, 129, 0, 255, 257, 300, 16]
    starts = np.concatenate([[3], 3 + np.cumsum(lens)]).astype(np.int32)
    total = int(starts[-1]) + 5
    (q, k, v), dev = _inputs(hq * 100 + d, total, hq, hkv, d, fused)
    scale = d ** -0.5
    got, status = _run(*dev, starts, scale)
    want, bound = chunks.prompts(q, k, v, starts, scale)
    assert status == 0
    _check(got, want, bound, slice(3, int(starts[-1])))
    assert (got[:3] == 7).all() and (got[int(starts[-1]):] == 7).all()


@pytest.mark.parametrize("hq,hkv,d,lens", [(4, 1, 128, [1031]), (2, 2, 128, [1500, 700]), (4, 2, 64, [2051]), (3, 1, 64, [900, 1, 640])])
def test_prompts_of_many_stages(hq, hkv, d, lens):
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, k, v), dev = _inputs(77 + d, int(starts[-1]), hq, hkv, d, True)
    got, status = _run(*dev, starts, d ** -0.5)
    want, bound = chunks.prompts(q, k, v, starts, d ** -0.5)
    assert status == 0
    _check(got, want, bound)


@pytest.mark.parametrize("hq,hkv,d", [(16, 8, 64), (8, 8, 128)])
def test_many_short_prompts(hq, hkv, d):
    """More units than CTAs, most of them a single stage that ends inside its box."""
    lens = [1 + 37 * i % 150 for i in range(150)]
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, k, v), dev = _inputs(6, int(starts[-1]), hq, hkv, d, True)
    got, status = _run(*dev, starts, d ** -0.5)
    want, bound = chunks.prompts(q, k, v, starts, d ** -0.5)
    assert status == 0
    _check(got, want, bound)


@pytest.mark.parametrize("size,scale", [(1.0, 2.0), (30.0, 0.088), (300.0, 0.088), (1e-20, 1.0), (1.0, 1e-30)])
def test_prompts_scores_of_any_size(size, scale):
    """One token takes all the weight, or all take the same."""
    starts = np.array([0, 200, 333], np.int32)
    (q, k, v), dev = _inputs(5, 333, 4, 2, 128, False, size)
    got, status = _run(*dev, starts, scale)
    want, bound = chunks.prompts(q, k, v, starts, np.float64(np.float32(scale)))
    assert status == 0
    _check(got, want, bound)


def test_prompts_growing_maxima():
    """Every stage's scores exceed the one's before it by far (the accumulator is rescaled each time), and the other way round."""
    import torch

    for sign in (1, -1):
        n, d = 700, 64
        (q, k, v), _ = _inputs(9, n, 2, 1, d, False)
        kf = widen(k) * 0.1
        kf[:, 0, 0] = sign * np.arange(n) * 0.5
        qf = widen(q) * 0.1
        qf[:, :, 0] = 3.0
        bits = lambda a: to_numpy(torch.tensor(a, dtype=torch.float32).to(torch.bfloat16))  # noqa: E731
        q, k = bits(qf), bits(kf)
        starts = np.array([0, n], np.int32)
        got, status = _run(to_torch(q), to_torch(k), to_torch(np.ascontiguousarray(v)), starts, 0.5)
        want, bound = chunks.prompts(q, k, v, starts, 0.5)
        assert status == 0
        _check(got, want, bound)


def test_prompts_see_nothing_of_their_neighbours():
    """NaN in every row before, between and behind the sequences in question."""
    starts = np.array([0, 50, 183, 190, 300], np.int32)
    (q, k, v), dev = _inputs(11, 310, 8, 2, 128, True)
    want, bound = chunks.prompts(q, k, v, starts, 0.1)
    import torch

    for keep in (1, 2, 3):
        mask = torch.ones(310, dtype=torch.bool, device="cuda")
        mask[starts[keep]:starts[keep + 1]] = False
        x = [t.clone() for t in dev]
        for t in x:
            t[mask] = float("nan")
        got, status = _run(*x, starts, 0.1)
        assert status == 0
        _check(got, want, bound, slice(starts[keep], starts[keep + 1]))


def test_prompts_flag_bad_lengths():
    import paged_kv_cache_280_gb300 as pa

    (q, k, v), dev = _inputs(12, 100, 4, 2, 64, False)
    want, bound = chunks.prompts(q, k, v, [0, 30, 60, 100], 0.1)
    for starts, most, bad in (([0, 30, 60, 101], 100, (60, 100)), ([0, 30, 60, 100], 35, (60, 100)), ([-1, 30, 60, 100], 100, (0, 30))):
        got, status = _run(*dev, np.array(starts), 0.1, max_len=most)
        assert status == pa.PA_DEV_BAD_SEQ_LEN
        a, b = bad
        assert (got[a:b] == 7).all()
        good = np.r_[0:a, b:100]
        _check(got, want, bound, good)
    got, status = _run(*dev, np.array([0, 60, 30, 100]), 0.1, max_len=100)  # a length of -30
    assert status == pa.PA_DEV_BAD_SEQ_LEN


def test_prompts_empty_calls():
    import torch

    (_, _, _), dev = _inputs(13, 10, 4, 2, 64, False)
    got, status = _run(*dev, np.zeros(4, np.int32), 0.1, max_len=0)
    assert status == 0 and (got == 7).all()
    got, status = _run(*dev, np.zeros(4, np.int32), 0.1, max_len=10)
    assert status == 0 and (got == 7).all()
    none = [t[:0] for t in dev]
    assert _run(*none, np.zeros(2, np.int32), 0.1, max_len=3)[1] == 0
    torch.cuda.synchronize()


def test_prompts_offsets_past_32_bits():
    import torch

    total, hq, hkv, d, row = 70000, 2, 1, 64, 40960  # 2.9 G elements from the first token to the last
    lens = [70000 - 400, 150, 250]
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    starts = starts[1:]  # the two at the end
    (q, k, v), dev = _inputs(14, 400, hq, hkv, d, False)
    big = torch.zeros(total * row, dtype=torch.bfloat16, device="cuda").view(total, row)
    views = []
    for i, t in enumerate(dev):
        h = t.shape[1]
        view = big[:, i * 4 * d:i * 4 * d + h * d].unflatten(1, (h, d))
        view[-400:] = t
        views.append(view)
    got, status = _run(*views, starts, 0.125)
    want, bound = chunks.prompts(q, k, v, starts - starts[0], 0.125)
    assert status == 0
    _check(got[-400:], want, bound)


def test_prompts_on_another_stream_captured_and_repeated():
    import torch
    import paged_kv_cache_280_gb300 as pa

    starts = np.array([0, 129, 400, 401], np.int32)
    _, (q, k, v) = _inputs(15, 401, 8, 2, 128, True)
    a, _ = _run(q, k, v, starts, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, _ = _run(q, k, v, starts, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    cu = to_torch(starts)
    out = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prompt_attention(out, q, k, v, cu, 271, 0.1)
    graph.replay()
    assert torch.equal(a, out)
    q.mul_(-1)
    a, _ = _run(q, k, v, starts, 0.1)
    graph.replay()
    assert torch.equal(a, out)


@pytest.mark.parametrize("hq,hkv,d", [(6, 2, 64), (8, 2, 128)])
def test_prompts_odd_strides_and_alignment(hq, hkv, d):
    """Token strides that are multiples of 16 bytes only, an output that is 16-byte aligned only, a loose bound on the lengths."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    lens = [130, 1, 77, 300]
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(starts[-1])
    host, dev = _inputs(77 + d, n, hq, hkv, d, False)
    spread = []
    for x, extra in zip(dev, (8, 24, 40)):
        wide = torch.full((n, x.shape[1] * d + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, : x.shape[1] * d] = x.flatten(1)
        spread.append(wide.as_strided(x.shape, (wide.shape[1], d, 1)))
    out = torch.full((n * hq * d + 8,), 7.0, dtype=torch.bfloat16, device="cuda")[8:].view(n, hq, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_prompt_attention(out, *spread, to_torch(starts), 1 << 30, d ** -0.5, status=status)
    assert status.item() == 0 and out.data_ptr() % 32 == 16
    _check(out, *chunks.prompts(*host, starts, d ** -0.5))


@pytest.mark.parametrize("hq,hkv,d,lens", [(16, 8, 128, [300] * 40), (16, 8, 64, [129, 300, 61, 500] * 12), (8, 8, 128, [270, 140] * 30)])
def test_prompts_many_units_to_a_cta(hq, hkv, d, lens):
    """Units of two tiles and of one behind one another in every CTA, tiles that see a stage less than their neighbour; equal
    calls give equal bits."""
    import torch

    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    host, dev = _inputs(900 + d + hq, int(starts[-1]), hq, hkv, d, True)
    got, status = _run(*dev, starts, d ** -0.5)
    assert status == 0
    _check(got, *chunks.prompts(*host, starts, d ** -0.5))
    for _ in range(20):
        again, status = _run(*dev, starts, d ** -0.5)
        assert status == 0 and torch.equal(again, got)


@pytest.mark.parametrize("where", [0, 300, 599])
def test_hundreds_of_prompts_with_a_long_one_and_a_loose_bound(where):
    lens = [(7 * i) % 40 for i in range(600)]
    lens[where] = 2500
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    host, dev = _inputs(1234 + where, int(starts[-1]), 2, 1, 64, False)
    got, status = _run(*dev, starts, 0.125, max_len=1 << 30)
    assert status == 0
    _check(got, *chunks.prompts(*host, starts, 0.125))
