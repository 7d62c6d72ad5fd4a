"""GPU: chunk attention over FP8 and 4-bit pools (pa_prefill_attention_fp8, _fp4) against the definition in float64."""
import numpy as np
import pytest

import synth
from gpu_cases import to_numpy, to_torch, widen
from oracle import chunks, kv4

pytestmark = pytest.mark.gpu


def _pool(rng, kind, nb, hkv, bs, d):
    if kind == "fp8":
        p = rng.integers(0, 0x48, (nb, hkv, bs, d)) | (rng.integers(0, 2, (nb, hkv, bs, d)) << 7)  # up to 4
        return p.astype(np.uint8)
    p = rng.integers(0, 256, (nb, hkv, bs * (d // 2 + d // 16)))
    p[:, :, bs * d // 2:] = rng.integers(0x20, 0x39, (nb, hkv, bs * d // 16))  # scales of 1 / 8 .. 1
    return p.astype(np.uint8)


class Case:
    def __init__(self, seed, kind, lens, news, hq, hkv, d, bs, size=1.0, poison=True, scale=None):
        rng = np.random.default_rng(seed)
        self.kind, self.hq, self.hkv, self.d, self.bs = kind, hq, hkv, d, bs
        self.lens, self.news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        need = -(-self.lens // bs)
        nb = int(need.sum()) + 4
        ids = rng.permutation(nb)
        self.tables = np.zeros((len(lens), max(1, int(need.max()))), np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = ids[at:at + n]
            at += n
        self.kp, self.vp = _pool(rng, kind, nb, hkv, bs, d), _pool(rng, kind, nb, hkv, bs, d)
        if poison:  # the slots of no token hold NaN
            used = np.zeros((nb, bs), bool)
            for b, n in enumerate(self.lens):
                t = np.arange(n)
                used[self.tables[b, t // bs], t % bs] = True
            for p in (self.kp, self.vp):
                if kind == "fp8":
                    p.transpose(0, 2, 1, 3)[~used] = 0x7F
                else:
                    kv4.split(p, d, bs)[1].transpose(0, 2, 1, 3)[~used] = 0x7F
        q = rng.standard_normal((max(1, int(self.starts[-1])), hq, d)).astype(np.float32) * np.float32(size)
        self.q = kv4.to_bf16(q)[: int(self.starts[-1])]
        self.ks, self.vs, self.scale = 0.37, 1.5, d ** -0.5 if scale is None else scale

    def device(self):
        self.dev = [to_torch(x) for x in (self.kp, self.vp, self.tables, self.lens, self.starts)]
        self.dq = to_torch(self.q)
        return self

    def run(self, workspace=None, max_q=None, stream=None, out=None):
        import torch
        import paged_kv_cache_280_gb300 as pa

        if not hasattr(self, "dev"):
            self.device()
        kp, vp, tables, lens, starts = self.dev
        most = int(self.news.max(initial=0)) if max_q is None else max_q
        if workspace is None:
            workspace = torch.zeros(pa.pa_prefill_workspace_bytes(most, self.hq, self.hkv, self.d), dtype=torch.uint8, device="cuda")
        if out is None:
            out = torch.full(self.dq.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        call = pa.pa_prefill_attention_fp8 if self.kind == "fp8" else pa.pa_prefill_attention_fp4
        call(out, self.dq, kp, vp, self.ks, self.vs, tables, lens, starts, most, self.scale, workspace, stream=stream)
        self.ws = workspace
        return out

    def status(self):
        import torch

        return int(self.ws[:4].view(torch.int32).item())

    def want(self, seqs=None):
        return chunks.chunks(self.q, self.kp, self.vp, self.kind, self.ks, self.vs, self.tables, self.lens, self.starts,
                             np.float64(np.float32(self.scale)), self.bs, seqs)

    def check(self, out, rows=None, seqs=None):
        want, bound = self.want(seqs)
        g = widen(to_numpy(out))
        if rows is not None:
            g, want, bound = g[rows], want[rows], bound[rows]
        assert np.all(np.isfinite(g))
        err, limit = np.abs(g - want), bound + 2.0 ** -8 * (np.abs(want) + bound) + 1e-30
        worst = np.unravel_index(np.argmax(err / limit), err.shape)
        assert np.all(err <= limit), f"max |err| {err.max():.3e}, {(err / limit).max():.2f} of the bound at {worst}"


KINDS = [("fp8", 128), ("fp4", 128), ("fp4", 64)]


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("hq,hkv,bs", [(8, 8, 16), (4, 2, 32), (6, 2, 16), (8, 2, 16), (5, 1, 32), (6, 1, 16), (14, 2, 16), (8, 1, 32)])
def test_chunks_ragged(kind, d, hq, hkv, bs):
    """No new token, one, a whole prompt, tails of longer contexts, several tiles; lengths around blocks and stages."""
    lens = [37, 1, 130, 64, 200, 90, 17, 128, 300, 256]
    news = [0, 1, 130, 20, 150, 9, 17, 1, 129, 128]
    c = Case(100 + hq + d + bs, kind, lens, news, hq, hkv, d, bs)
    c.check(c.run())
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("lens,news,hq,hkv", [([4097], [5], 8, 2), ([9000, 129, 5000], [1, 129, 3], 8, 1), ([3000], [3000], 2, 1),
                                              ([2500, 2500], [300, 40], 4, 4), ([20000], [17], 4, 1)])
def test_chunks_split_over_long_contexts(kind, d, lens, news, hq, hkv):
    c = Case(200 + sum(lens) % 97 + d, kind, lens, news, hq, hkv, d, 16)
    c.check(c.run())
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_many_sequences(kind, d):
    """More sequences than a warp has lanes, without new tokens here and there, and runs of them."""
    lens = [1 + 53 * i % 400 for i in range(150)]
    news = [0 if i % 7 == 0 or 40 <= i < 75 else 1 + (29 * i) % min(n, 70) for i, n in enumerate(lens)]
    c = Case(250 + d, kind, lens, news, 4, 2, d, 16)
    c.check(c.run())
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_single_tokens_match_the_decode(kind, d):
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(300 + d, kind, [1, 16, 17, 250, 33, 1300], [1] * 6, 8, 2, d, 16)
    got = c.run()
    c.check(got)
    kp, vp, tables, lens, _ = c.dev
    out = torch.empty_like(c.dq)
    ws = torch.zeros(pa.pa_decode_workspace_bytes(6, 8, 2, d), dtype=torch.uint8, device="cuda")
    decode = pa.pa_decode_attention_fp8 if kind == "fp8" else pa.pa_decode_attention_fp4
    decode(out, c.dq, kp, vp, c.ks, c.vs, tables, lens, 1300, c.scale, ws)
    want, bound = c.want()  # both within it, so within twice of each other
    assert np.all(np.abs(widen(to_numpy(out)) - widen(to_numpy(got))) <= 2 * (bound + 2.0 ** -8 * (np.abs(want) + bound)) + 2.0 ** -11 * np.abs(want))


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("size,scale", [(1.0, 3.0), (60.0, 0.1), (1e30, 1e-31), (1e-30, 1e29), (1.0, 1e-25)])
def test_chunks_scores_of_any_size(kind, d, size, scale):
    c = Case(400 + d, kind, [300, 140], [60, 140], 4, 2, d, 16, size=size, scale=scale)
    c.check(c.run())
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_rows_of_unequal_elements(kind, d):
    """One query element far above the others, rows of zeros."""
    c = Case(410 + d, kind, [300, 140], [60, 140], 4, 2, d, 16)
    q = widen(c.q).astype(np.float32)
    q[:, :, 3] *= 1000
    q[5] = 0
    q[7, 1] = 0
    c.q = kv4.to_bf16(q)
    c.check(c.run())


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_flag_bad_sequences_and_blocks(kind, d):
    import paged_kv_cache_280_gb300 as pa

    c = Case(500 + d, kind, [40, 10, 70], [12, 11, 70], 8, 2, d, 16)  # sequence 1: 11 new tokens of 10
    out = c.run(max_q=300)
    assert c.status() == pa.PA_DEV_BAD_SEQ_LEN
    good = np.r_[0:12, 23:93]
    c.check(out, rows=good, seqs=[0, 2])
    assert (out[12:23] == 7).all()
    c = Case(501 + d, kind, [40, 10, 70], [12, 5, 70], 8, 2, d, 16)
    out = c.run(max_q=69)
    assert c.status() == pa.PA_DEV_BAD_SEQ_LEN and (out[17:] == 7).all()
    c.check(out, rows=np.r_[0:17], seqs=[0, 1])
    c = Case(502 + d, kind, [40, 20, 70], [12, 5, 70], 8, 2, d, 16)
    c.lens = c.lens.copy()
    c.lens[1] = 16 * c.tables.shape[1] + 1
    out = c.run()
    assert c.status() == pa.PA_DEV_BAD_SEQ_LEN and (out[12:17] == 7).all()
    c.check(out, rows=np.r_[0:12, 17:87], seqs=[0, 2])
    for bad in (-1, 1 << 30):
        c = Case(503 + d, kind, [40, 20, 70], [12, 5, 70], 8, 2, d, 16)
        c.tables = c.tables.copy()
        c.tables[1, 1] = bad
        out = c.run()
        assert c.status() == pa.PA_DEV_BAD_BLOCK_ID
        c.check(out, rows=np.r_[0:12, 17:87], seqs=[0, 2])


@pytest.mark.parametrize("kind,d", KINDS)
def test_one_workspace_for_calls_of_many_shapes(kind, d):
    """Call after call on one workspace, each as on a fresh one, bit for bit, and again."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    cases = [Case(600, kind, [4000, 100], [3, 100], 8, 1, d, 16), Case(601, kind, [700] * 5, [200] * 5, 4, 4, d, 32),
             Case(602, kind, [1], [1], 1, 1, d, 16), Case(603, kind, [9000], [33], 6, 2, d, 16)]
    alone = [c.run().clone() for c in cases]
    ws = torch.zeros(max(pa.pa_prefill_workspace_bytes(int(c.news.max()), c.hq, c.hkv, d) for c in cases), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c, want in zip(cases, alone):
            assert torch.equal(c.run(ws), want)
    for c in cases:
        c.check(c.run(ws))
    assert cases[0].status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("byte", [0xFF, 0x7F])
def test_a_workspace_may_hold_anything_behind_its_status_word(kind, d, byte):
    import torch
    import paged_kv_cache_280_gb300 as pa

    for c in (Case(610, kind, [4000, 700], [3, 500], 8, 2, d, 16), Case(611, kind, [40], [1], 1, 1, d, 32)):
        want = c.run().clone()
        ws = torch.full((pa.pa_prefill_workspace_bytes(int(c.news.max()), c.hq, c.hkv, d),), byte, dtype=torch.uint8, device="cuda")
        ws[:4] = 0
        assert torch.equal(c.run(ws), want) and c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("lens,news,hq,hkv", [([2500, 2500], [300, 40], 4, 4), ([700] * 5, [200] * 5, 4, 4), ([9000, 129], [1, 129], 8, 1)])
def test_chunks_repeat_bit_for_bit(kind, d, lens, news, hq, hkv):
    """The same call many times over: whichever CTA ends last, and however the roles of a CTA interleave."""
    import torch

    c = Case(650 + d, kind, lens, news, hq, hkv, d, 16)
    want = c.run()
    c.check(want)
    out = torch.empty_like(want)
    for _ in range(100):
        assert torch.equal(c.run(c.ws, out=out), want)


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_on_another_stream_and_captured(kind, d):
    import torch

    c = Case(700 + d, kind, [3000, 140, 20], [20, 140, 1], 8, 2, d, 16)
    a = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros_like(c.ws)
    out, b = torch.zeros_like(a), torch.zeros_like(a)
    torch.cuda.synchronize()
    c.run(ws, stream=side, out=b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws, out=out)
    graph.replay()
    assert torch.equal(a, out)
    c.dq.mul_(-1)
    a = c.run()
    graph.replay()
    graph.replay()
    assert torch.equal(a, out)


@pytest.mark.parametrize("kind,d", KINDS)
def test_chunks_pools_past_32_bits(kind, d):
    """Blocks beyond 4 GiB of a pool."""
    import torch

    c = Case(800 + d, kind, [150, 40], [30, 40], 4, 2, d, 16, poison=False).device()
    rec = c.dev[0][0].numel()
    shift = (1 << 32) // rec + 3
    big = [torch.zeros((shift + len(p), *p.shape[1:]), dtype=torch.uint8, device="cuda") for p in c.dev[:2]]
    for b, p in zip(big, c.dev[:2]):
        b[shift:] = p
    c.dev[:2] = big
    c.dev[2] = c.dev[2] + shift
    c.check(c.run())
    assert c.status() == 0


def test_nothing_to_do():
    c = Case(900, "fp8", [40, 30], [0, 0], 4, 2, 128, 16)
    assert c.run(max_q=0).shape[0] == 0
    c = Case(901, "fp4", [40, 0], [1, 0], 4, 2, 128, 16)
    c.check(c.run())


def test_small_workspace_is_refused():
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(902, "fp8", [40, 30], [3, 4], 4, 2, 128, 16)
    need = pa.pa_prefill_workspace_bytes(4, 4, 2, 128)
    with pytest.raises(pa.PAError, match="WORKSPACE_TOO_SMALL"):
        c.run(torch.zeros(need - 16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("lens,news,hkv,max_q", [([9 + 5 * i % 17 for i in range(20)], [1] * 20, 4, None),
                                                 ([1 + 7 * i % 90 for i in range(48)], [1] * 48, 8, 500),
                                                 ([30 + 41 * i % 900 for i in range(32)], [1 + i % 3 for i in range(32)], 8, None)])
def test_many_short_units(kind, d, lens, news, hkv, max_q):
    """More units than CTAs or nearly so, each a stage or a few; in slots of two tiles too."""
    c = Case(700 + d + len(lens), kind, lens, news, hkv, hkv, d, 32)
    c.check(c.run(max_q=max_q))
    assert c.status() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_two_graphs_at_once_and_an_output_aligned_to_16_bytes(kind, d):
    """Captured calls on workspaces of their own, replayed on two streams at once, again and again."""
    import torch

    cases = [Case(800, kind, [5000, 70], [6, 70], 8, 2, d, 16).device(), Case(801, kind, [900, 2100], [300, 40], 4, 4, d, 32).device()]
    want = [c.run().clone() for c in cases]
    outs = [torch.zeros(w.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(w.shape) for w in want]
    graphs, streams = [], [torch.cuda.Stream() for _ in cases]
    for c, out, s in zip(cases, outs, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(c.ws, out=out)
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, out, w in zip(cases, outs, want):
        assert out.data_ptr() % 32 == 16 and torch.equal(out, w) and c.status() == 0
        c.check(out)


@pytest.mark.parametrize("kind,d", KINDS)
def test_the_longest_sequences_are_refused(kind, d):
    """Lengths whose last stage would pass 31 bits, over a table that is wide enough: flagged, their rows not written."""
    import torch
    import paged_kv_cache_280_gb300 as pa

    c = Case(820, kind, [40, 33], [1, 2], 1, 1, d, 16).device()
    want = c.run().clone()
    table = torch.zeros((2, 1 << 27), dtype=torch.int32, device="cuda")
    table[:, : c.tables.shape[1]] = c.dev[2]
    for length in (2 ** 31 - 1, 2 ** 31 - 255):
        c.dev[2], c.dev[3] = table, torch.tensor([length, 33], dtype=torch.int32, device="cuda")
        got = c.run()
        assert c.status() == pa.PA_DEV_BAD_SEQ_LEN
        assert (got[0] == 7.0).all() and torch.equal(got[1:], want[1:])
