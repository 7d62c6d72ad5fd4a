"""The checks of the rotating append and of the 4-bit entry points: bad calls come back from the host (no GPU needed)."""
import ctypes

import pytest

import paged_kv_cache_280_gb300 as pa

FAKE = ctypes.c_void_p(1 << 20)  # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
INVALID, UNSUPPORTED = 1, 2


def _rope(**kw):
    a = dict(q_out=FAKE, q=FAKE, qs=8 * 128, k=FAKE, ks=2 * 128, v=FAKE, vs=2 * 128, pos=FAKE, table=FAKE, maxp=100, rot=128,
             inter=0, kp=FAKE, vp=FAKE, slots=FAKE, n=4, hq=8, hkv=2, d=128, bs=16, nb=10, dt=pa.PA_BF16, pdt=pa.PA_BF16,
             ksc=1.0, vsc=1.0, status=None, stream=None)
    a["q_out"] = ctypes.c_void_p(1 << 21)
    a.update(kw)
    return pa._lib.pa_rope_and_cache(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), 0), (dict(n=-1), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID), (dict(maxp=0), INVALID),
    (dict(rot=0), INVALID), (dict(rot=144), INVALID), (dict(rot=24), UNSUPPORTED), (dict(inter=2), INVALID),
    (dict(rot=48, pdt=pa.PA_FP4_E2M1), UNSUPPORTED), (dict(dt=pa.PA_FP8_E4M3), UNSUPPORTED),
    (dict(pdt=pa.PA_F32), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(d=64, rot=64, pdt=pa.PA_FP8_E4M3), UNSUPPORTED), (dict(pdt=7), UNSUPPORTED),
    (dict(ksc=0.0), INVALID), (dict(vsc=float("nan")), INVALID), (dict(ksc=float("inf")), INVALID), (dict(vsc=-1.0), INVALID),
    (dict(qs=8 * 128 - 8), INVALID), (dict(ks=2 * 128 + 4), INVALID), (dict(vs=0), INVALID), (dict(vs=-256), INVALID),
    (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID), (dict(pos=None), INVALID),
    (dict(table=None), INVALID), (dict(slots=None), INVALID), (dict(kp=None), INVALID), (dict(vp=ODD), INVALID),
    (dict(q=ODD), INVALID), (dict(table=ODD), INVALID), (dict(pos=ctypes.c_void_p((1 << 20) + 2)), INVALID),
    (dict(slots=ctypes.c_void_p((1 << 20) + 4)), INVALID), (dict(status=ctypes.c_void_p((1 << 20) + 1)), INVALID),
    (dict(q_out=FAKE, qs=12 * 128), INVALID),  # in place, but not laid out as q_out is
    (dict(n=1 << 29), UNSUPPORTED),
])
def test_rope_refusals(kw, want):
    assert _rope(**kw) == want


def _append(**kw):
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, slots=FAKE, n=4, hkv=2, d=128, bs=16, nb=10, dt=pa.PA_BF16, ks=1.0, vs=1.0,
             status=None, stream=None)
    a.update(kw)
    return pa._lib.pa_reshape_and_cache_fp4(*a.values())


def _unpack(**kw):
    a = dict(kp=FAKE, vp=FAKE, blocks=FAKE, n=4, ko=FAKE, vo=FAKE, hkv=2, d=128, bs=16, nb=10, dt=pa.PA_BF16, ks=1.0, vs=1.0,
             status=None, stream=None)
    a.update(kw)
    return pa._lib.pa_unpack_blocks_fp4(*a.values())


@pytest.mark.parametrize("call", [_append, _unpack])
@pytest.mark.parametrize("kw,want", [
    (dict(n=0), 0), (dict(n=-1), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID), (dict(dt=pa.PA_FP8_E4M3), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(ks=0.0), INVALID), (dict(vs=float("inf")), INVALID),
    (dict(kp=None), INVALID), (dict(vp=ODD), INVALID),
])
def test_append_and_unpack_refusals(call, kw, want):
    assert call(**kw) == want


def test_append_and_unpack_pointer_refusals():
    assert _append(k=None) == INVALID and _append(v=ODD) == INVALID and _append(slots=ctypes.c_void_p((1 << 20) + 4)) == INVALID
    assert _unpack(blocks=None) == INVALID and _unpack(ko=ODD) == INVALID and _unpack(vo=None) == INVALID
    assert _append(n=1 << 30, hkv=4) == UNSUPPORTED and _unpack(hkv=1 << 25) == UNSUPPORTED


def _decode(**kw):
    a = dict(out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, ks=1.0, vs=1.0, tables=FAKE, mb=4, lens=FAKE, msl=64, b=2, hq=8, hkv=2, d=128,
             bs=16, nb=10, scale=0.1, part=0, ws=FAKE, wsb=1 << 24, stream=None)
    a.update(kw)
    return pa._lib.pa_decode_attention_fp4(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(b=0), INVALID), (dict(hq=7), INVALID), (dict(hq=18), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(bs=8), UNSUPPORTED),
    (dict(ks=0.0), INVALID), (dict(vs=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(part=24), INVALID),
    (dict(part=-16), INVALID), (dict(msl=-1), INVALID), (dict(mb=0), INVALID), (dict(nb=0), INVALID), (dict(q=None), INVALID),
    (dict(kp=ODD), INVALID), (dict(out=ODD), INVALID), (dict(ws=None), INVALID), (dict(lens=None), INVALID),
    (dict(nb=1 << 30), UNSUPPORTED),
])
def test_decode_refusals(kw, want):
    assert _decode(**kw) == want


def test_planned_decode_needs_a_plan():
    assert pa._lib.pa_decode_attention_fp4_planned(FAKE, FAKE, FAKE, FAKE, 1.0, 1.0, FAKE, 4, FAKE, 64, 2, 8, 2, 128, 16, 10, 0.1,
                                                   0, FAKE, 1 << 24, None, 0, None) == INVALID


def test_whole_block_copies_check_the_4_bit_pool():
    args = [FAKE, FAKE, FAKE, 0, 2, 128, 16, 10, pa.PA_FP4_E2M1, None, None]
    assert pa._lib.pa_copy_blocks(*args) == 0  # nothing to copy
    assert pa._lib.pa_copy_blocks(*args[:5], 96, *args[6:]) == UNSUPPORTED
    assert pa._lib.pa_copy_blocks(*args[:8], 4, *args[9:]) == UNSUPPORTED
    assert pa._lib.pa_swap_out(FAKE, FAKE, FAKE, 1, ODD, FAKE, 2, 64, 32, 10, pa.PA_FP4_E2M1, None, None) == INVALID


def test_binding_refusals():
    """The binding refuses what the C side cannot see: CPU tensors, wrong types, pools that hold no whole rows."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 128)
    pool = torch.zeros(5, 2, pa.fp4_block_bytes(128, 16), dtype=torch.uint8)
    slots, ids = torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_new must be a CUDA"):
        pa.pa_reshape_and_cache_fp4(k, k, pool, pool, slots, 1.0, 1.0)
    with pytest.raises(pa.PAError, match="whole rows"):
        pa.pa_reshape_and_cache_fp4(k, k, pool[..., :100], pool, slots, 1.0, 1.0)
    with pytest.raises(pa.PAError, match="uint8"):
        pa.pa_decode_attention_fp4(k, k, pool.float(), pool, 1.0, 1.0, slots, slots, 1, 1.0, pool)
    with pytest.raises(ValueError, match="out must be a CUDA"):
        pa.pa_decode_attention_fp4(k, k, pool, pool, 1.0, 1.0, ids[None], ids, 1, 1.0, pool)
    with pytest.raises(ValueError, match="k_pool must be a CUDA"):
        pa.pa_unpack_blocks_fp4(pool, pool, ids, torch.zeros(3, 2, 16, 128), torch.zeros(3, 2, 16, 128), 1.0, 1.0)
    with pytest.raises(ValueError, match="k must be a CUDA"):
        pa.pa_rope_and_cache(None, None, k, k, ids, k[0], pool, pool, slots)
    with pytest.raises(pa.PAError, match="go together"):
        pa.pa_rope_and_cache(None, k, k, k, ids, k[0], pool, pool, slots)
    with pytest.raises(pa.PAError):
        pa.pa_copy_blocks(torch.zeros(5, 2, 100, dtype=torch.uint8), pool, torch.zeros(1, 2, dtype=torch.int32))
    assert pa._token_rows(torch.zeros(4, 12, 64)[:, 2:5], "k") == 12 * 64 and pa._token_rows(torch.zeros(1, 3, 64), "k") == 192
    for bad in (torch.zeros(4, 64, 3).transpose(1, 2), torch.zeros(4, 3, 64)[:, ::2]):
        with pytest.raises(ValueError, match="contiguous heads"):
            pa._token_rows(bad, "k")


class _On:
    """A tensor's face: what the binding asks of one."""

    def __init__(self, device, dtype, shape, contiguous=True):
        self.device_, self.dtype, self.shape, self.contiguous, self.is_cuda = device, dtype, shape, contiguous, device >= 0

    def get_device(self):
        return self.device_

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return 1

    def data_ptr(self):
        return 1 << 20


def test_tensor_checks():
    assert pa._ptr(_On(0, "f", (2, 3)), "f", (2, 3), 0, "x") == 1 << 20
    for bad, error, text in ((_On(1, "f", (2, 3)), ValueError, "x is on cuda:1, but the current device is cuda:0"),
                             (_On(-1, "f", (2, 3)), ValueError, "x must be a CUDA tensor"),
                             (_On(0, "g", (2, 3)), pa.PAError, "expected f"), (_On(0, "f", (2, 4)), pa.PAError, "expected"),
                             (_On(0, "f", (2, 3), False), ValueError, "contiguous")):
        with pytest.raises(error, match=text):
            pa._ptr(bad, "f", (2, 3), 0, "x")
    assert pa._rows_ptr(_On(0, "f", (2, 3), False), "f", (2, 3), 0, "x") == 1 << 20
    with pytest.raises(ValueError, match="current device"):
        pa._rows_ptr(_On(1, "f", (2, 3)), "f", (2, 3), 0, "x")
    torch = pytest.importorskip("torch")
    assert pa._status_ptr(None, 0) is None and pa._status_ptr(_On(0, torch.int32, (1,)), 0) == 1 << 20
    with pytest.raises(pa.PAError):
        pa._status_ptr(_On(0, torch.int64, (1,)), 0)
