"""The binding's shared tables under two threads."""
import types

import pytest

import paged_kv_cache_280_gb300 as pa


def test_a_second_thread_during_the_first_lookup(monkeypatch):
    """The table of dtypes is filled on first use.  A thread that comes in between finds it empty or whole: here the second
    lookup is made while the first one is filling it, at the moment it asks for the FP8 type."""
    torch = pytest.importorskip("torch")
    seen = []

    class Torch(types.SimpleNamespace):
        def __getattr__(self, name):  # not in the namespace: the FP8 type, asked for by name
            if name != "float8_e4m3fn":
                raise AttributeError(name)
            if not seen:
                seen.append(None)
                for dtype, code in ((torch.float8_e4m3fn, pa.PA_FP8_E4M3), (torch.bfloat16, pa.PA_BF16)):
                    seen.append((pa._dtype_code(types.SimpleNamespace(dtype=dtype)), code))
            return torch.float8_e4m3fn

    monkeypatch.setattr(pa, "_dtype_codes", {})
    monkeypatch.setattr(pa, "_torch", lambda: Torch(float32=torch.float32, bfloat16=torch.bfloat16, uint8=torch.uint8))
    assert pa._dtype_code(types.SimpleNamespace(dtype=torch.float32)) == pa.PA_F32
    assert len(seen) == 3 and all(got == code for got, code in seen[1:])
    with pytest.raises(pa.PAError):
        pa._dtype_code(types.SimpleNamespace(dtype=torch.float64))
