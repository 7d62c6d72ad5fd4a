"""The rotating append and the 4-bit KV cache of paged_kv_cache_280_gb300: what is measured.

Four operators over a paged key-value cache (blocks of 16 or 32 token slots, scattered in a pool):

- the rotating append: queries and keys are rotated by their positions, keys and values go to their slots;
- the 4-bit append: keys and values are quantised to E2M1 codes with an E4M3 scale per 16 elements;
- the unpacking of 4-bit blocks into dense bf16 or fp32 blocks, in the layout that the prefill reads;
- decode attention of one new token per sequence over a 4-bit cache.

A 4-bit pool is a uint8 tensor [num_blocks][Hkv][bs * (D / 2 + D / 16)].  The record of one block and
head holds the codes of its bs token rows (D / 2 bytes each, element 2 j in the low half of byte j), then
their scale bytes (D / 16 each).  Value = E2M1(code) * E4M3(scale byte) * pool scale.
"""
import math

import torch

own = False  # True: the framework's kernels; False: the plain forms

BF16, F32 = "bf16", "f32"
MAX_POS = 40960  # rows of the cos / sin table
GROUP = 16  # elements per E4M3 scale


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _rope(name, n, hq, hkv, d, bs, dtype, pool, rot, inter, fused, pad, scatter):
    return {"name": name, "kind": "rope", "n": n, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "in": dtype, "pool": pool,
            "rot": rot, "inter": inter, "fused": fused, "pad": pad, "scatter": scatter}


def _append(name, n, hkv, d, bs, dtype, out, pad, scatter):
    return {"name": name, "kind": "append4", "n": n, "hkv": hkv, "d": d, "bs": bs, "in": dtype, "out": out,
            "pad": pad, "scatter": scatter}


def _unpack(name, blocks, hkv, d, bs, out):
    return {"name": name, "kind": "unpack4", "blocks": blocks, "hkv": hkv, "d": d, "bs": bs, "out": out}


def _decode(name, b, hq, hkv, d, bs, lo, hi, empty, part):
    return {"name": name, "kind": "decode4", "b": b, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "lo": lo, "hi": hi,
            "empty": empty, "part": part}


def listed():
    return [
        # one decoding user: the latency of the step's first kernel
        _rope("rope_one_token", 1, 32, 8, 128, 16, BF16, BF16, 128, False, True, 0, True),
        # a serving batch into FP8 pools, some rows of the captured batch unused (padding)
        _rope("rope_fp8_batch", 256, 32, 32, 128, 16, BF16, "fp8", 128, False, True, 7, True),
        # a prompt chunk: q, k and v are views of one fused projection
        _rope("rope_chunk", 8191, 64, 8, 128, 16, BF16, BF16, 128, False, True, 0, False),
        # fp32, rotation of the first half of each head only, adjacent pairs
        _rope("rope_f32_partial", 2053, 16, 4, 64, 32, F32, F32, 32, True, False, 5, False),
        # a prompt chunk into the 4-bit cache, read back for the chunk's prefill
        _rope("rope_fp4_chunk", 4099, 32, 8, 128, 16, BF16, "fp4", 128, False, True, 0, False),
        # one token per sequence of a batch, appended to the 4-bit cache; the blocks read back
        _append("append4_batch", 256, 32, 128, 16, BF16, BF16, 3, True),
        # a long prompt's keys and values
        _append("append4_chunk", 16383, 8, 128, 32, BF16, BF16, 0, False),
        # the context of a 128 K-token conversation, unpacked for the prefill of its next turn
        _unpack("unpack4_context", 8192, 8, 128, 16, BF16),
        # one user, a page of context
        _decode("decode4_one_user", 1, 32, 8, 128, 16, 1031, 1031, False, 0),
        # a serving batch of mixed lengths, 4 query heads per KV head
        _decode("decode4_gqa4_batch", 64, 32, 8, 128, 16, 32, 4095, True, 0),
        # many heads, one query head each
        _decode("decode4_mha_batch", 256, 32, 32, 128, 16, 32, 4095, False, 0),
        # four very long contexts, split into parts of 2048 tokens
        _decode("decode4_long", 4, 64, 8, 128, 32, 131072, 131072, False, 2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "append4", "unpack4", "decode4", "decode4"])
    hkv, d, bs = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128, 128]), rng.choice([16, 32])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    dtype = rng.choice([BF16, BF16, F32])
    if kind == "rope":
        pool = rng.choice([dtype, "fp4"] + (["fp8"] if d == 128 else []))
        n = _log_int(rng, 1, max(1, min(8191, 600000 // ((g + 2) * hkv))))
        c = _rope("", n, g * hkv, hkv, d, bs, dtype, pool, rng.choice([d, d, d // 2]), rng.random() < 0.4,
                  rng.random() < 0.6, n // 16 if rng.random() < 0.5 else 0, n * hkv < 24000 and rng.random() < 0.5)
    elif kind == "append4":
        n = _log_int(rng, 1, min(16383, 130000 // hkv))
        c = _append("", n, hkv, d, bs, dtype, rng.choice([BF16, F32]), n // 9 if rng.random() < 0.5 else 0, n * hkv < 24000 and rng.random() < 0.5)
    elif kind == "unpack4":
        c = _unpack("", _log_int(rng, 1, min(4095, 65536 * 16 // (hkv * bs) // 2)), hkv, d, bs, rng.choice([BF16, F32]))
    else:
        b = _log_int(rng, 1, 200)
        top = max(2, min(100000, 6000000 // (b * hkv)))
        hi = _log_int(rng, 2, top)
        part = rng.choice([0, 0, 0, 256, 1024])
        c = _decode("", b, g * hkv, hkv, d, bs, max(1, int(hi * rng.random())), hi, b > 2 and rng.random() < 0.5, part)
    del c["name"]
    return c


def _lens(case):
    """The case's lengths: even steps of the logarithm between lo and hi; the first is empty where the case says so."""
    b, lo, hi = case["b"], case["lo"], case["hi"]
    lens = [int(round(lo * (hi / lo) ** ((i + 0.5) / b))) for i in range(b)] if hi > lo else [hi] * b
    if b > 1:
        lens[-1] = hi
    if case["empty"]:
        lens[0] = 0
    return lens


def _size(dtype):
    return {BF16: 2, F32: 4, "fp8": 1, "fp4": 0.5 + 1 / GROUP}[dtype]


def work(case):
    k, d, hkv = case["kind"], case["d"], case["hkv"]
    if k == "rope":
        n = case["n"] - case["pad"]
        rows = n * (case["hq"] + 2 * hkv) * d * _size(case["in"])
        out = n * (case["hq"] * _size(case["in"]) + 2 * hkv * _size(case["pool"])) * d
        bytes_ = rows + out + 12 * case["n"] + 4 * case["rot"] * min(n, MAX_POS)
        if case["pool"] == "fp4":  # the written blocks are read back
            bytes_ += 2 * _blocks_written(case) * case["bs"] * hkv * d * (_size("fp4") + 2)
        return {"bytes": bytes_, "flops": 3 * n * (case["hq"] + hkv) * case["rot"]}
    if k == "append4":
        n = case["n"] - case["pad"]
        bytes_ = 2 * n * hkv * d * (_size(case["in"]) + _size("fp4")) + 8 * case["n"]
        bytes_ += 2 * _blocks_written(case) * case["bs"] * hkv * d * (_size("fp4") + _size(case["out"]))
        return {"bytes": bytes_, "flops": 6 * n * hkv * d}
    if k == "unpack4":
        return {"bytes": 2 * case["blocks"] * case["bs"] * hkv * d * (_size("fp4") + _size(case["out"])) + 4 * case["blocks"],
                "flops": 4 * case["blocks"] * case["bs"] * hkv * d}
    tokens = sum(_lens(case))
    blocks = sum(-(-t // case["bs"]) for t in _lens(case))
    return {"bytes": 2 * tokens * hkv * d * _size("fp4") + 2 * case["b"] * case["hq"] * d * 2 + 4 * blocks + 4 * case["b"],
            "flops": 4 * tokens * case["hq"] * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _blocks_written(case):
    """Blocks that the case's tokens lie in: one each where they are scattered, else a run."""
    return case["n"] if case["scatter"] else -(-case["n"] // case["bs"])


def _slots(case, g):
    """(blocks int32, slots int64): the tokens' blocks in a scattered pool; padding tokens get slot -1."""
    n, bs, nb = case["n"], case["bs"], _blocks_written(case)
    num_blocks = nb + max(2, nb // 10)
    blocks = torch.randperm(num_blocks, generator=g, device="cuda")[:nb]
    i = torch.arange(n, device="cuda")
    if case["scatter"]:
        slots = blocks * bs + torch.randint(0, bs, (n,), generator=g, device="cuda")
    else:
        slots = blocks[i // bs] * bs + i % bs
    if case["pad"]:
        slots[torch.randperm(n, generator=g, device="cuda")[: case["pad"]]] = -1
    return num_blocks, blocks.to(torch.int32), slots


def _dtype(name):
    return {BF16: torch.bfloat16, F32: torch.float32}[name]


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(_dtype(dtype))


def _random_pool4(g, num_blocks, hkv, bs, d):
    """A 4-bit pool of any codes, with scales between 1/4 and 1."""
    p = torch.randint(0, 256, (num_blocks, hkv, bs * (d // 2 + d // GROUP)), generator=g, device="cuda", dtype=torch.uint8)
    p[:, :, bs * d // 2:] = torch.randint(0x28, 0x39, (num_blocks, hkv, bs * d // GROUP), generator=g, device="cuda", dtype=torch.uint8)
    return p


def _cos_sin(rot):
    """cos | sin of position * 10000^(-2 j / rot) [MAX_POS][rot], the angles in 64 bits."""
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s, d, hkv, bs = dict(case), case["d"], case["hkv"], case["bs"]
    # powers of two and not: the pools' fp32 scales, as a calibration leaves them
    s["ks"], s["vs"] = 0.043, 0.0625
    s["kst"], s["vst"] = (torch.full((1,), x, device="cuda") for x in (s["ks"], s["vs"]))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["kind"] in ("rope", "append4"):
        n = case["n"]
        hq = case.get("hq", 0)
        s["num_blocks"], s["blocks"], s["slots"] = _slots(case, g)
        pool = case.get("pool", "fp4")
        if case["kind"] == "append4" or not case["fused"]:
            s["q"], s["k"], s["v"] = (_randn(g, (n, h, d), case["in"]) for h in (hq, hkv, hkv))
        else:
            qkv = _randn(g, (n, hq + 2 * hkv, d), case["in"])
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if case["kind"] == "rope":
            s["cos_sin"] = _cos_sin(case["rot"])
            if case["scatter"]:
                s["pos"] = torch.randint(0, MAX_POS, (n,), generator=g, device="cuda", dtype=torch.int32)
            else:
                first = int(torch.randint(0, MAX_POS - n + 1, (1,), generator=g, device="cuda"))
                s["pos"] = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
            s["q_out"] = torch.zeros((n, hq, d), device="cuda", dtype=_dtype(case["in"]))
        for p in ("kp", "vp"):
            if pool == "fp4":
                s[p] = _random_pool4(g, s["num_blocks"], hkv, bs, d)
            elif pool == "fp8":
                s[p] = _randn(g, (s["num_blocks"], hkv, bs, d), F32).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                s[p] = _randn(g, (s["num_blocks"], hkv, bs, d), pool)
        if pool == "fp4":
            s["out_dtype"] = _dtype(case.get("out", BF16))
    elif case["kind"] == "unpack4":
        num_blocks = case["blocks"] + max(2, case["blocks"] // 10)
        s["blocks"] = torch.randperm(num_blocks, generator=g, device="cuda")[: case["blocks"]].to(torch.int32)
        s["kp"], s["vp"] = (_random_pool4(g, num_blocks, hkv, bs, d) for _ in range(2))
        s["out_dtype"] = _dtype(case["out"])
    else:
        lens = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
        s["lens"] = lens[torch.randperm(case["b"], generator=g, device="cuda")].contiguous()
        need = (s["lens"].long() + bs - 1) // bs
        mb = -(-case["hi"] // bs)
        num_blocks = int(need.sum()) + max(2, int(need.sum()) // 10)
        perm = torch.randperm(num_blocks, generator=g, device="cuda")
        at = torch.cumsum(need, 0) - need
        col = torch.arange(mb, device="cuda")
        inside = col[None] < need[:, None]
        s["tables"] = torch.where(inside, perm[(at[:, None] + col[None]).clamp(max=num_blocks - 1)], 0).to(torch.int32)
        s["q"] = _randn(g, (case["b"], case["hq"], d), BF16)
        s["kp"], s["vp"] = (_random_pool4(g, num_blocks, hkv, bs, d) for _ in range(2))
        # scores of standard deviation about 1, as trained heads have them
        s["ks"], s["vs"] = 0.5, 0.5
        s["kst"], s["vst"] = (torch.full((1,), 0.5, device="cuda") for _ in range(2))
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.zeros((case["b"], case["hq"], d), device="cuda", dtype=torch.bfloat16)
        s["workspace"] = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    if "out_dtype" in s:
        shape = (len(s["blocks"]), hkv, bs, d)
        s["k_out"], s["v_out"] = (torch.empty(shape, device="cuda", dtype=s["out_dtype"]) for _ in range(2))
    return s


# ---------------------------------------------------------------------------
# the plain forms: elementary torch operations in fp32
# ---------------------------------------------------------------------------

def _rotate(x, cos, sin, rot, inter):
    """x [N][H][D] fp32, cos / sin [N][1][rot / 2] fp32."""
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if inter:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
    else:
        y[..., : rot // 2], y[..., rot // 2: rot] = ra, rb
    return y


def _quantise4(x, scale):
    """x [..][D] fp32 -> (packed codes [..][D / 2], scale bytes [..][D / 16])."""
    y = (x / scale).unflatten(-1, (-1, GROUP))
    s = (y.abs().amax(-1, keepdim=True) / torch.full_like(scale, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()
    z = (y / torch.where(sf == 0, 1.0, sf)).abs() * (sf != 0)
    # midpoints of the E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    code = (z > 0.25).to(torch.uint8) + (z >= 0.75) + (z > 1.25) + (z >= 1.75) + (z > 2.5) + (z >= 3.5) + (z > 5.0)
    code = (code + 8 * (torch.signbit(y) & (sf != 0)).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8).squeeze(-1)


def _values4(pool, bs, d):
    """A 4-bit pool's values without the pool scale, fp32 [num_blocks][Hkv][bs][D]."""
    codes = pool[..., : bs * d // 2].unflatten(-1, (bs, d // 2))
    scales = pool[..., bs * d // 2:].unflatten(-1, (bs, d // GROUP)).contiguous().view(torch.float8_e4m3fn).float()
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=pool.device)
    lut = torch.cat([mags, -mags])
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, GROUP)) * scales[..., None]).flatten(-2)


def _plain_store(s, pool, x, scale, slots, blk, off):
    kind, bs, d = s.get("pool", "fp4"), s["bs"], s["d"]
    if kind == "fp4":
        codes, scales = _quantise4(x, scale)
        pool[..., : bs * d // 2].unflatten(-1, (bs, d // 2))[blk, :, off] = codes
        pool[..., bs * d // 2:].unflatten(-1, (bs, d // GROUP))[blk, :, off] = scales
    elif kind == "fp8":
        pool[blk, :, off] = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool[blk, :, off] = x.to(pool.dtype)


def _plain_append(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    blk, off = at // s["bs"], at % s["bs"]
    k, v = s["k"].float(), s["v"].float()
    if s["kind"] == "rope":
        cs = s["cos_sin"][s["pos"]][:, None]
        cos, sin = cs[..., : s["rot"] // 2], cs[..., s["rot"] // 2:]
        k = _rotate(k, cos, sin, s["rot"], s["inter"])
        q = _rotate(s["q"].float(), cos, sin, s["rot"], s["inter"]).to(s["q"].dtype)
        s["q_out"].copy_(torch.where(keep[:, None, None], q, s["q_out"]))
    _plain_store(s, s["kp"], k[keep], s["kst"], at, blk, off)
    _plain_store(s, s["vp"], v[keep], s["vst"], at, blk, off)


def _plain_unpack(s):
    at = s["blocks"].long()
    for pool, out, scale in ((s["kp"], s["k_out"], s["kst"]), (s["vp"], s["v_out"], s["vst"])):
        out.copy_(_values4(pool[at], s["bs"], s["d"]) * scale)


def _plain_decode(s):
    b, hkv, d, bs = s["b"], s["hkv"], s["d"], s["bs"]
    at = s["tables"].long()
    t = at.shape[1] * bs
    seen = (torch.arange(t, device="cuda")[None] < s["lens"][:, None])[:, None, None]  # [B][1][1][T]
    q = s["q"].float().view(b, hkv, -1, d)
    k = (_values4(s["kp"], bs, d) * s["kst"])[at].transpose(1, 2).reshape(b, hkv, t, d)
    x = (q @ k.transpose(2, 3)) * s["scale"]
    del k
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(x - m), 0.0)
    v = (_values4(s["vp"], bs, d) * s["vst"])[at].transpose(1, 2).reshape(b, hkv, t, d)
    o = (p @ v) / p.sum(-1, keepdim=True)
    s["out"].copy_(torch.where(s["lens"][:, None, None] > 0, o.view(b, -1, d), 0.0))


def run(s):
    kind = s["kind"]
    if own:
        import paged_kv_cache_280_gb300 as pa

        if kind == "rope":
            pa.pa_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["kp"], s["vp"], s["slots"],
                                 interleaved=s["inter"], k_scale=s["ks"], v_scale=s["vs"], status=s["status"])
        elif kind == "append4":
            pa.pa_reshape_and_cache_fp4(s["k"], s["v"], s["kp"], s["vp"], s["slots"], s["ks"], s["vs"],
                                        status=s["status"])
        elif kind == "decode4":
            pa.pa_decode_attention_fp4(s["out"], s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["tables"], s["lens"],
                                       s["hi"], s["scale"], s["workspace"], partition_tokens=s["part"])
        if "k_out" in s:
            pa.pa_unpack_blocks_fp4(s["kp"], s["vp"], s["blocks"], s["k_out"], s["v_out"], s["ks"], s["vs"],
                                    status=s["status"])
    else:
        if kind in ("rope", "append4"):
            _plain_append(s)
        elif kind == "decode4":
            _plain_decode(s)
        if "k_out" in s:
            _plain_unpack(s)
    return _outputs(s)


def _outputs(s):
    """What the pass computed: the pools as the values that they hold (4-bit ones unpacked by the pass itself)."""
    r = {}
    if s["kind"] == "decode4":
        return {"out": s["out"]}
    if s["kind"] == "rope":
        r["q"] = s["q_out"]
    if "k_out" in s:
        r["k"], r["v"] = s["k_out"], s["v_out"]
    else:
        r["k"], r["v"] = ((p.view(torch.float8_e4m3fn) if s["pool"] == "fp8" else p) for p in (s["kp"], s["vp"]))
    return r


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token where the plain form works on whole tensors
# ---------------------------------------------------------------------------

def _e4m3(byte):
    """Values of E4M3 bytes from their fields: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = byte.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, (e - 7).double()), m / 512)
    return torch.where(b >= 128, -mag, mag)


def _e2m1(code):
    """Values of E2M1 codes from their fields: sign, 2 exponent bits (bias 1), 1 mantissa bit."""
    c = code.long()
    e, m = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, (e - 1).double()), m / 2)
    return torch.where(c >= 8, -mag, mag)


def _block64(pool, blocks, bs, d):
    """float64 [n][Hkv][bs][D] of the blocks of a 4-bit pool, without the pool scale."""
    r = pool[blocks.long()]
    n, hkv = r.shape[:2]
    c = r[..., : bs * d // 2].reshape(n, hkv, bs, d // 2)
    f = _e4m3(r[..., bs * d // 2:].reshape(n, hkv, bs, d // GROUP))
    v = torch.empty((n, hkv, bs, d), dtype=torch.float64, device=pool.device)
    v[..., 0::2], v[..., 1::2] = _e2m1(c & 15), _e2m1(c >> 4)
    return v * f.repeat_interleave(GROUP, -1)


def _nearest(x, grid):
    """Nearest value of an ascending grid of magnitudes; a tie goes to the even index.  x >= 0, float64."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), grid[lo], grid[hi])


def _store64(kind, x, scale):
    """What a pool reads back for float64 x, with the fp32 quotients that the stored format is defined by."""
    if kind in (BF16, F32):
        return x
    grid8 = _e4m3(torch.arange(127, device=x.device))
    y = (x.float().double() / scale).float().double()
    if kind == "fp8":
        return _nearest(y.abs(), grid8) * torch.sign(y)
    y = y.unflatten(-1, (-1, GROUP))
    s = _nearest((y.abs().amax(-1, keepdim=True) / 6).float().double(), grid8)
    z = (y / torch.where(s == 0, 1.0, s)).float().double()
    grid4 = _e2m1(torch.arange(8, device=x.device))
    return (_nearest(z.abs(), grid4) * torch.sign(z) * s).flatten(-2) * scale


def exact(case, seed):
    s = prepare(case, seed)
    d, bs, hkv = case["d"], case["bs"], case["hkv"]
    ks, vs = s["kst"].double(), s["vst"].double()
    if case["kind"] == "unpack4":
        return {"k": _block64(s["kp"], s["blocks"], bs, d) * ks, "v": _block64(s["vp"], s["blocks"], bs, d) * vs}
    if case["kind"] == "decode4":
        out = torch.zeros((case["b"], case["hq"], d), dtype=torch.float64, device="cuda")
        group = case["hq"] // hkv
        for i, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            table = s["tables"][i, : -(-n // bs)]
            for h in range(0, hkv, 4):  # a few heads at a time: very long contexts
                kb = _block64(s["kp"][:, h:h + 4], table, bs, d)
                vb = _block64(s["vp"][:, h:h + 4], table, bs, d)
                kb, vb = (t.movedim(0, 1).reshape(t.shape[1], -1, d)[:, :n] for t in (kb, vb))
                q = s["q"][i, h * group: (h + kb.shape[0]) * group].double().view(kb.shape[0], group, d)
                p = torch.softmax(torch.einsum("hgd,htd->hgt", q, kb) * (ks * s["scale"]), -1)
                out[i, h * group: (h + kb.shape[0]) * group] = (torch.einsum("hgt,htd->hgd", p, vb) * vs).reshape(-1, d)
        return {"out": out}
    pool = case.get("pool", "fp4")
    new = {"k": s["k"].double(), "v": s["v"].double()}
    r = {}
    if case["kind"] == "rope":
        half = case["rot"] // 2
        cs = s["cos_sin"].double()[s["pos"].long()]
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
        turned = {}
        for name in ("q", "k"):
            x = s[name].double()
            y = x.clone()
            y[..., a] = x[..., a] * cs[:, None, :half] - x[..., b] * cs[:, None, half:]
            y[..., b] = x[..., b] * cs[:, None, :half] + x[..., a] * cs[:, None, half:]
            turned[name] = y
        new["k"] = turned["k"]
        r["q"] = torch.where((s["slots"] >= 0)[:, None, None], turned["q"], 0.0)
    kept = (s["slots"] >= 0).nonzero().flatten()
    slot = s["slots"][kept]
    for name, pooled, scale in (("k", s["kp"], ks), ("v", s["vp"], vs)):
        if pool == "fp4":
            every = torch.arange(pooled.shape[0], device="cuda")
            full = torch.zeros((pooled.shape[0], hkv, bs, d), dtype=torch.float64, device="cuda")
            full[s["blocks"].long()] = _block64(pooled, every[s["blocks"].long()], bs, d) * scale
        elif pool == "fp8":
            full = _e4m3(pooled)
        else:
            full = pooled.double()
        full[slot // bs, :, slot % bs] = _store64(pool, new[name][kept], scale)
        r[name] = full[s["blocks"].long()] if pool == "fp4" else full
    return r
