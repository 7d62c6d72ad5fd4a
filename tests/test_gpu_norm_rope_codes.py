"""GPU: the codes and scales that the normed rotating append stores in quantised pools, byte for byte.

Over fp32 inputs the dense turned keys hold exactly the fp32 values that are quantised, so the oracle's quantiser has to give the
pool from them.  Over bf16 inputs the same fp32 values are formed from the same numbers, so the pool is that of the inputs widened."""
import numpy as np
import pytest

import synth
from gpu_cases import to_numpy, to_torch
from oracle import kv4
from test_gpu_norm_rope import EPS
from test_gpu_rope import MAXP, _inputs, _oracle_append, _pool

pytestmark = pytest.mark.gpu

CASES = [
    # n, hq, hkv, d, bs, pool, rot, interleaved, fused, k_scale
    (1, 2, 1, 128, 16, "fp8", 128, False, True, 0.037),
    (61, 16, 2, 128, 32, "fp8", 64, True, False, 0.037),
    (61, 4, 4, 128, 16, "fp8", 128, False, True, 1e-3),   # most values saturate
    (61, 4, 4, 128, 16, "fp8", 48, False, False, 30.0),   # among the smallest codes
    (1, 1, 1, 64, 32, "fp4", 64, True, False, 0.037),
    (61, 12, 4, 128, 32, "fp4", 96, False, True, 0.037),
    (61, 6, 6, 64, 16, "fp4", 32, True, True, 1e-4),      # scales saturate
    (61, 6, 3, 128, 16, "fp4", 128, False, False, 40.0),  # among the smallest scales
    (900, 8, 8, 64, 32, "fp4", 64, False, True, 1.0 / 2688),
    (900, 24, 8, 128, 16, "fp8", 128, True, True, 1.0 / 64),
]


def _append(q, k, v, w, pos, table, pools, slots, inter, ks, vs):
    import torch
    import paged_kv_cache_280_gb300 as pa

    q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(k.shape, dtype=k.dtype, device="cuda")
    pa.pa_norm_rope_and_cache(q_out, k_out, q, k, v, *w, EPS, pos, table, *pools, slots, interleaved=inter, k_scale=ks, v_scale=vs)
    return k_out


@pytest.mark.parametrize("n,hq,hkv,d,bs,pool,rot,inter,fused,ks", CASES)
def test_stored_keys_are_the_quantised_dense_keys(n, hq, hkv, d, bs, pool, rot, inter, fused, ks):
    seed, vs = 7000 + n + hq + d + rot, 0.21
    (_, _, v), dev = _inputs(seed, n, hq, hkv, d, "f32", fused)
    nb = -(-n // bs) + 2
    slots = synth.permutation(seed, nb * bs)[:n].astype(np.int64)
    pos = synth.uniform_ints(seed + 1, n, 0, MAXP - 1).astype(np.int32)
    rng = np.random.default_rng(seed)
    w = [to_torch(rng.uniform(-2, 2, d).astype(np.float32)) for _ in range(2)]
    if n > 5:
        slots[[3, n - 2]] = -1
        dev[1][5] = 0  # a row of zeros
        dev[1][7, 0, :40] *= 1000
    table = kv4.cos_sin_table(MAXP, rot)
    kp, vp = _pool(seed, nb, hkv, bs, d, pool), _pool(seed + 7, nb, hkv, bs, d, pool)
    pools = [to_torch(kp), to_torch(vp)]
    k_out = _append(*dev, w, to_torch(pos), to_torch(table), pools, to_torch(slots), inter, ks, vs)
    _oracle_append(pool, kp, vp, to_numpy(k_out), v, slots, bs, ks, vs)
    assert np.array_equal(to_numpy(pools[0]), kp) and np.array_equal(to_numpy(pools[1]), vp)


@pytest.mark.parametrize("n,hq,hkv,d,bs,pool,rot,inter,fused,ks", CASES)
def test_keys_of_bf16_and_the_same_in_fp32_are_stored_alike(n, hq, hkv, d, bs, pool, rot, inter, fused, ks):
    import torch

    seed, vs = 8000 + n + hq + d + rot, 0.21
    _, dev = _inputs(seed, n, hq, hkv, d, "bf16", fused)
    nb = -(-n // bs) + 2
    slots, pos = synth.permutation(seed, nb * bs)[:n].astype(np.int64), synth.uniform_ints(seed + 1, n, 0, MAXP - 1).astype(np.int32)
    rng = np.random.default_rng(seed)
    w = [to_torch(rng.uniform(-2, 2, d).astype(np.float32)) for _ in range(2)]
    rest = (w, to_torch(pos), to_torch(kv4.cos_sin_table(MAXP, rot)))
    pools = [[to_torch(_pool(seed + i, nb, hkv, bs, d, pool)) for i in range(2)] for _ in range(2)]
    narrow = _append(*dev, *rest, pools[0], to_torch(slots), inter, ks, vs)
    wide = _append(*(t.float() for t in dev), *rest, pools[1], to_torch(slots), inter, ks, vs)
    assert torch.equal(narrow, wide.to(torch.bfloat16))
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
