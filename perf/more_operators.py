"""Normed rotating append, prompt attention and chunk attention over quantised pools: what is measured.

Four operators of a serving step with a paged key-value cache (blocks of 16 or 32 token slots, scattered in a pool):

- the normed rotating append: queries and keys are divided by their head's root mean square, weighted, turned by their
  positions; keys and values go to their slots, the turned keys also to a dense buffer where a prompt attention follows;
- prompt attention: whole prompts of different lengths, packed one behind the other, each token sees its own prompt up to itself;
- chunk attention over FP8 pools: the last tokens of each sequence see its whole cached context up to themselves;
- the same over 4-bit pools.

An FP8 pool is uint8 E4M3 codes [num_blocks][Hkv][bs][D] with one pool scale.  A 4-bit pool is a uint8 tensor
[num_blocks][Hkv][bs * (D / 2 + D / 16)]: the record of one block and head holds the codes of its bs token rows (D / 2 bytes
each, element 2 j in the low half of byte j), then their scale bytes (D / 16 each).  Value = E2M1(code) * E4M3(scale byte) *
pool scale.
"""
import math

import torch

own = False  # True: the framework's kernels; False: the plain forms

BF16, F32 = "bf16", "f32"
MAX_POS = 40960  # rows of the cos / sin table
GROUP = 16  # elements per E4M3 scale
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm_rope(name, n, hq, hkv, d, bs, dtype, pool, rot, inter, fused, keys, pad, scatter):
    return {"name": name, "kind": "norm_rope", "n": n, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "in": dtype, "pool": pool,
            "rot": rot, "inter": inter, "fused": fused, "keys": keys, "pad": pad, "scatter": scatter}


def _prompt(name, b, hq, hkv, d, lo, hi, empty, fused, pad):
    return {"name": name, "kind": "prompt", "b": b, "hq": hq, "hkv": hkv, "d": d, "lo": lo, "hi": hi, "empty": empty,
            "fused": fused, "pad": pad}


def _chunk(name, pool, b, hq, hkv, d, bs, new_lo, new_hi, lo, hi, empty):
    return {"name": name, "kind": "chunk", "pool": pool, "b": b, "hq": hq, "hkv": hkv, "d": d, "bs": bs, "new_lo": new_lo,
            "new_hi": new_hi, "lo": lo, "hi": hi, "empty": empty}


def listed():
    return [
        # one decoding user: the latency of the step's first kernel
        _norm_rope("normrope_one_token", 1, 32, 8, 128, 16, BF16, BF16, 128, False, True, False, 0, True),
        # a prompt chunk into FP8 pools; the turned keys are kept for the prompt's own attention
        _norm_rope("normrope_fp8_chunk", 8191, 64, 8, 128, 16, BF16, "fp8", 128, False, True, True, 0, False),
        # fp32, adjacent pairs of half of each head, into the 4-bit cache, some rows of the batch unused; read back
        _norm_rope("normrope_f32_fp4", 2053, 16, 4, 64, 32, F32, "fp4", 32, True, False, False, 5, False),
        # a batch of short prompts of a small model, one of them empty, rows behind the last prompt unused
        _prompt("prompt_ragged", 24, 16, 4, 64, 1, 1031, True, False, 7),
        # a serving batch of equal prompts
        _prompt("prompt_batch", 16, 32, 8, 128, 1031, 1031, False, True, 0),
        # one long prompt of a large model
        _prompt("prompt_long", 1, 64, 8, 128, 8191, 8191, False, True, 0),
        # the check of 5 drafted tokens per sequence: few rows over long contexts
        _chunk("chunk8_verify", "fp8", 32, 32, 8, 128, 16, 5, 5, 1024, 16383, False),
        # the next turns of four conversations, a query head per key head
        _chunk("chunk8_turn", "fp8", 4, 32, 32, 128, 32, 129, 517, 2048, 16383, False),
        # one user, a few words on a page of context
        _chunk("chunk4_one_user", "fp4", 1, 32, 8, 128, 16, 17, 17, 1031, 1031, False),
        # drafted tokens over two very long contexts
        _chunk("chunk4_long", "fp4", 2, 64, 8, 128, 32, 4, 9, 131072, 131072, False),
        # a document added to a long conversation
        _chunk("chunk4_turn", "fp4", 1, 32, 8, 128, 16, 2047, 2047, 32767, 32767, False),
        # a mixed batch of a small model: single tokens, chunks, and a sequence without new tokens
        _chunk("chunk4_mixed", "fp4", 12, 16, 4, 64, 16, 1, 130, 131, 4095, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["norm_rope", "norm_rope", "prompt", "prompt", "chunk", "chunk", "chunk"])
    hkv, d, bs = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128, 128]), rng.choice([16, 32])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if kind == "norm_rope":
        dtype = rng.choice([BF16, BF16, F32])
        pool = rng.choice([dtype, "fp4"] + (["fp8"] if d == 128 else []))
        n = _log_int(rng, 1, max(1, min(8191, 600000 // ((g + 2) * hkv))))
        c = _norm_rope("", n, g * hkv, hkv, d, bs, dtype, pool, rng.choice([d, d, d // 2]), rng.random() < 0.4,
                       rng.random() < 0.6, rng.random() < 0.5, n // 16 if rng.random() < 0.5 else 0,
                       n * hkv < 24000 and rng.random() < 0.5)
    elif kind == "prompt":
        b = _log_int(rng, 1, 48)
        top = min(8191, int(math.sqrt(4.0e9 / (b * g * hkv))))
        hi = _log_int(rng, 1, max(1, top))
        c = _prompt("", b, g * hkv, hkv, d, max(1, int(hi * rng.random())), hi, b > 2 and rng.random() < 0.4,
                    rng.random() < 0.5, rng.choice([0, 0, 3]))
    else:
        pool = rng.choice(["fp4", "fp8"])
        d = 128 if pool == "fp8" else d
        b = _log_int(rng, 1, 48)
        hi = _log_int(rng, 2, max(2, min(131072, 4000000 // (b * hkv))))
        new_hi = _log_int(rng, 1, max(1, min(hi, 2047, int(2.0e9 / (b * g * hkv * hi)))))
        c = _chunk("", pool, b, g * hkv, hkv, d, bs, max(1, int(new_hi * rng.random())), new_hi,
                   max(new_hi, int(hi * rng.random())), hi, b > 2 and rng.random() < 0.5)
    del c["name"]
    return c


def _spread(b, lo, hi):
    """b sizes at even steps of the logarithm between lo and hi, the last one hi."""
    sizes = [int(round(lo * (hi / lo) ** ((i + 0.5) / b))) for i in range(b)] if hi > lo else [hi] * b
    return sizes[:-1] + [hi]


def _lens(case):
    """Contexts of a chunk case, lengths of a prompt case (the first is empty where the case says so)."""
    lens = _spread(case["b"], case["lo"], case["hi"])
    if case["kind"] == "prompt" and case["empty"]:
        lens[0] = 0
    return lens


def _news(case):
    """New tokens of each sequence of a chunk case; longer chunks go to the shorter contexts."""
    news = _spread(case["b"], case["new_lo"], case["new_hi"])[::-1]
    if case["empty"]:
        news[0] = 0
    return [min(n, t) for n, t in zip(news, _lens(case))]


def _size(dtype):
    return {BF16: 2, F32: 4, "fp8": 1, "fp4": 0.5 + 1 / GROUP}[dtype]


def work(case):
    k, d, hq, hkv = case["kind"], case["d"], case["hq"], case["hkv"]
    if k == "norm_rope":
        n = case["n"] - case["pad"]
        rows = n * (hq + 2 * hkv) * d * _size(case["in"])
        out = n * (hq * _size(case["in"]) + 2 * hkv * _size(case["pool"])) * d
        bytes_ = rows + out + 12 * case["n"] + 4 * case["rot"] * min(n, MAX_POS) + 8 * d
        if case["keys"]:
            bytes_ += n * hkv * d * _size(case["in"])
        if case["pool"] == "fp4":  # the written blocks are read back
            bytes_ += 2 * _blocks_written(case) * case["bs"] * hkv * d * (_size("fp4") + 2)
        return {"bytes": bytes_, "flops": n * (hq + hkv) * (4 * d + 3 * case["rot"])}
    if k == "prompt":
        lens = _lens(case)
        return {"bytes": sum(lens) * (2 * hq + 2 * hkv) * d * 2 + 4 * (case["b"] + 1),
                "flops": sum(n * (n + 1) // 2 for n in lens) * 4 * d * hq}
    lens, news = _lens(case), _news(case)
    read = sum(t for t, n in zip(lens, news) if n)
    blocks = sum(-(-t // case["bs"]) for t, n in zip(lens, news) if n)
    return {"bytes": 2 * read * hkv * d * _size(case["pool"]) + sum(news) * 2 * hq * d * 2 + 4 * blocks + 12 * case["b"],
            "flops": sum(n * (t - n) + n * (n + 1) // 2 for t, n in zip(lens, news)) * 4 * d * hq}


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


def _random_pool(g, kind, num_blocks, hkv, bs, d):
    """A pool of any codes; the 4-bit groups' scales between 1/4 and 1."""
    if kind == "fp8":
        return _randn(g, (num_blocks, hkv, bs, d), F32).to(torch.float8_e4m3fn).view(torch.uint8)
    if kind != "fp4":
        return _randn(g, (num_blocks, hkv, bs, d), kind)
    p = torch.randint(0, 256, (num_blocks, hkv, bs * (d // 2 + d // GROUP)), generator=g, device="cuda", dtype=torch.uint8)
    p[:, :, bs * d // 2:] = torch.randint(0x28, 0x39, (num_blocks, hkv, bs * d // GROUP), generator=g, device="cuda", dtype=torch.uint8)
    return p


def _cos_sin(rot):
    """cos | sin of position * 10000^(-2 j / rot) [MAX_POS][rot], the angles in 64 bits."""
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-2 * j / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _starts(sizes):
    return torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)


def _tables(g, lens, bs):
    """(num_blocks, block tables int32 [B][most]): each sequence's blocks, scattered in the pool."""
    need = (lens.long() + bs - 1) // bs
    most, total = int(need.max()), int(need.sum())
    num_blocks = total + max(2, total // 10)
    perm = torch.randperm(num_blocks, generator=g, device="cuda")
    col = torch.arange(most, device="cuda")
    at = (torch.cumsum(need, 0) - need)[:, None] + col
    return num_blocks, torch.where(col < need[:, None], perm[at.clamp(max=num_blocks - 1)], 0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s, d, hq, hkv = dict(case), case["d"], case["hq"], case["hkv"]
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["kind"] == "norm_rope":
        n, bs, pool = case["n"], case["bs"], case["pool"]
        s["num_blocks"], s["blocks"], s["slots"] = _slots(case, g)
        # projections: every token and head at a size of its own
        x = _randn(g, (n, hq + 2 * hkv, d), F32) * torch.exp(_randn(g, (n, hq + 2 * hkv, 1), F32))
        x[:, hq + hkv:] = _randn(g, (n, hkv, d), F32)
        x = x.to(_dtype(case["in"]))
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not case["fused"]:
            s["q"], s["k"], s["v"] = (s[t].contiguous() for t in "qkv")
        s["qw"], s["kw"] = (0.5 + torch.rand(d, generator=g, device="cuda") for _ in range(2))
        s["cos_sin"] = _cos_sin(case["rot"])
        if case["scatter"]:
            s["pos"] = torch.randint(0, MAX_POS, (n,), generator=g, device="cuda", dtype=torch.int32)
        else:
            first = int(torch.randint(0, MAX_POS - n + 1, (1,), generator=g, device="cuda"))
            s["pos"] = torch.arange(first, first + n, device="cuda", dtype=torch.int32)
        s["q_out"] = torch.zeros((n, hq, d), device="cuda", dtype=x.dtype)
        s["k_out"] = torch.zeros((n, hkv, d), device="cuda", dtype=x.dtype) if case["keys"] else None
        s["kp"], s["vp"] = (_random_pool(g, pool, s["num_blocks"], hkv, bs, d) for _ in range(2))
        # the pools' fp32 scales, as a calibration leaves them: no power of two, and one
        s["ks"], s["vs"] = 0.043, 0.0625
        if pool == "fp4":
            s["k_read"], s["v_read"] = (torch.empty((len(s["blocks"]), hkv, bs, d), device="cuda", dtype=torch.bfloat16)
                                        for _ in range(2))
    elif case["kind"] == "prompt":
        lens = _lens(case)
        order = torch.randperm(case["b"], generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["starts"], s["most"], total = _starts(lens), max(lens), sum(lens) + case["pad"]
        if case["fused"]:
            x = _randn(g, (total, hq + 2 * hkv, d), BF16)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (_randn(g, (total, h, d), BF16) for h in (hq, hkv, hkv))
        s["out"] = torch.zeros((total, hq, d), device="cuda", dtype=torch.bfloat16)
    else:
        bs, lens, news = case["bs"], _lens(case), _news(case)
        order = torch.randperm(case["b"], generator=g, device="cuda").tolist()
        news = [news[i] for i in order]
        s["lens"] = torch.tensor([lens[i] for i in order], dtype=torch.int32, device="cuda")
        s["starts"], s["most"] = _starts(news), max(news)
        num_blocks, s["tables"] = _tables(g, s["lens"], bs)
        s["kp"], s["vp"] = (_random_pool(g, case["pool"], num_blocks, hkv, bs, d) for _ in range(2))
        s["q"] = _randn(g, (sum(news), hq, d), BF16)
        # scores of standard deviation about 1, as trained heads have them
        s["ks"], s["vs"] = (0.5, 0.5) if case["pool"] == "fp4" else (0.875, 0.043)
        s["out"] = torch.zeros((sum(news), hq, d), device="cuda", dtype=torch.bfloat16)
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")  # of the largest call, kept by the program
    if "ks" in s:
        s["kst"], s["vst"] = (torch.full((1,), x, device="cuda") for x in (s["ks"], s["vs"]))
    s["scale"] = 1.0 / math.sqrt(d)
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


def _normed(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w


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


def _plain_store(s, pool, x, scale, blk, off):
    kind, bs, d = s["pool"], s["bs"], s["d"]
    if kind == "fp4":
        codes, scales = _quantise4(x, scale)
        pool[..., : bs * d // 2].unflatten(-1, (bs, d // 2))[blk, :, off] = codes
        pool[..., bs * d // 2:].unflatten(-1, (bs, d // GROUP))[blk, :, off] = scales
    elif kind == "fp8":
        pool[blk, :, off] = (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        pool[blk, :, off] = x.to(pool.dtype)


def _plain_norm_rope(s):
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    blk, off = at // s["bs"], at % s["bs"]
    cs = s["cos_sin"][s["pos"]][:, None]
    cos, sin = cs[..., : s["rot"] // 2], cs[..., s["rot"] // 2:]
    q = _rotate(_normed(s["q"].float(), s["qw"]), cos, sin, s["rot"], s["inter"])
    k = _rotate(_normed(s["k"].float(), s["kw"]), cos, sin, s["rot"], s["inter"])
    s["q_out"].copy_(torch.where(keep[:, None, None], q.to(s["q"].dtype), s["q_out"]))
    if s["keys"]:
        s["k_out"].copy_(torch.where(keep[:, None, None], k.to(s["k"].dtype), s["k_out"]))
    _plain_store(s, s["kp"], k[keep], s["kst"], blk, off)
    _plain_store(s, s["vp"], s["v"][keep].float(), s["vst"], blk, off)
    if s["pool"] == "fp4":
        blocks = s["blocks"].long()
        for pool, out, scale in ((s["kp"], s["k_read"], s["kst"]), (s["vp"], s["v_read"], s["vst"])):
            out.copy_(_values4(pool[blocks], s["bs"], s["d"]) * scale)


def _attend(q, k, v, seen, scale):
    """q [B][N][Hq][D], k / v [B][Hkv][T][D], seen [B][N][T] -> [B][N][Hq][D], all fp32; a row that sees nothing is NaN."""
    b, n, hq, d = q.shape
    hkv, t = k.shape[1:3]
    x = q.view(b, n, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d) @ k.transpose(2, 3)
    x = torch.where(seen[:, None, None], x.view(b, hkv, -1, n, t) * scale, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, -1, t) @ v).view(b, hkv, -1, n, d) / total
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)


def _padded(s):
    """(token index [B][most], its validity) of packed rows."""
    i = torch.arange(s["most"], device="cuda")[None]
    first, last = s["starts"][:-1, None].long(), s["starts"][1:, None].long()
    return (first + i).clamp(max=len(s["q"]) - 1), first + i < last


def _plain_prompt(s):
    at, valid = _padded(s)
    i = torch.arange(s["most"], device="cuda")
    seen = (i[None] <= i[:, None])[None] & valid[:, :, None]
    k, v = (s[x][at].float().transpose(1, 2) for x in "kv")
    v = torch.where(valid[:, None, :, None], v, 0.0)
    s["out"][at[valid]] = _attend(s["q"][at].float(), k, v, seen, s["scale"])[valid].to(s["out"].dtype)


def _plain_chunk(s):
    at, valid = _padded(s)
    tables, bs, d = s["tables"].long(), s["bs"], s["d"]
    t = torch.arange(tables.shape[1] * bs, device="cuda")
    first = s["lens"][:, None] - (s["starts"][1:] - s["starts"][:-1])[:, None]
    pos = first + torch.arange(s["most"], device="cuda")[None]
    seen = (t[None, None] <= pos[:, :, None]) & valid[:, :, None]
    held = (t[None] < s["lens"][:, None])[:, None, :, None]
    k, v = (((_values4(p[tables], bs, d) if s["pool"] == "fp4" else p[tables].view(torch.float8_e4m3fn).float()) * scale)
            .transpose(1, 2).flatten(2, 3) for p, scale in ((s["kp"], s["kst"]), (s["vp"], s["vst"])))
    v = torch.where(held, v, 0.0)
    s["out"][at[valid]] = _attend(s["q"][at].float(), k, v, seen, s["scale"])[valid].to(s["out"].dtype)


def run(s):
    kind = s["kind"]
    if own:
        import paged_kv_cache_280_gb300 as pa

        if kind == "norm_rope":
            pa.pa_norm_rope_and_cache(s["q_out"], s["k_out"], s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["pos"],
                                      s["cos_sin"], s["kp"], s["vp"], s["slots"], interleaved=s["inter"], k_scale=s["ks"],
                                      v_scale=s["vs"], status=s["status"])
            if s["pool"] == "fp4":
                pa.pa_unpack_blocks_fp4(s["kp"], s["vp"], s["blocks"], s["k_read"], s["v_read"], s["ks"], s["vs"],
                                        status=s["status"])
        elif kind == "prompt":
            pa.pa_prompt_attention(s["out"], s["q"], s["k"], s["v"], s["starts"], s["most"], s["scale"], status=s["status"])
        else:
            call = pa.pa_prefill_attention_fp4 if s["pool"] == "fp4" else pa.pa_prefill_attention_fp8
            call(s["out"], s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["tables"], s["lens"], s["starts"], s["most"],
                 s["scale"], s["workspace"])
    elif kind == "norm_rope":
        _plain_norm_rope(s)
    elif kind == "prompt":
        _plain_prompt(s)
    else:
        _plain_chunk(s)
    return _outputs(s)


def _outputs(s):
    """What the pass computed: the pools as the values that they hold (4-bit ones unpacked by the pass itself)."""
    if s["kind"] != "norm_rope":
        return {"out": s["out"]}
    r = {"q": s["q_out"]}
    if s["keys"]:
        r["keys"] = s["k_out"]
    if s["pool"] == "fp4":
        r["k"], r["v"] = s["k_read"], s["v_read"]
    else:
        r["k"], r["v"] = ((p.view(torch.float8_e4m3fn) if s["pool"] == "fp8" else p) for p in (s["kp"], s["vp"]))
    return r


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence and head by head where the plain form works on whole tensors
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


def _block64(pool, kind, blocks, bs, d):
    """float64 [n][H][bs][D] of the blocks of a quantised pool, without the pool scale."""
    r = pool[blocks.long()]
    if kind == "fp8":
        return _e4m3(r)
    n, h = r.shape[:2]
    c = r[..., : bs * d // 2].reshape(n, h, bs, d // 2)
    f = _e4m3(r[..., bs * d // 2:].reshape(n, h, bs, d // GROUP))
    v = torch.empty((n, h, bs, d), dtype=torch.float64, device=pool.device)
    v[..., 0::2], v[..., 1::2] = _e2m1(c & 15), _e2m1(c >> 4)
    return v * f.repeat_interleave(GROUP, -1)


def _nearest(x, grid):
    """Nearest value of an ascending grid of magnitudes; a tie goes to the even index.  x >= 0, float64."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), grid[lo], grid[hi])


def _store64(kind, x, scale):
    """What a pool reads back for float64 x."""
    if kind in (BF16, F32):
        return x
    grid8 = _e4m3(torch.arange(127, device=x.device))
    y = x / scale
    if kind == "fp8":
        return _nearest(y.abs(), grid8) * torch.sign(y)
    y = y.unflatten(-1, (-1, GROUP))
    s = _nearest(y.abs().amax(-1, keepdim=True) / 6, grid8)
    z = y / torch.where(s == 0, 1.0, s)
    grid4 = _e2m1(torch.arange(8, device=x.device))
    return (_nearest(z.abs(), grid4) * torch.sign(z) * s).flatten(-2) * scale


def _rows64(q, k, v, first, scale):
    """One key head: q [G][n][D], k / v [T][D], row i at position first + i."""
    x = torch.einsum("gnd,td->gnt", q, k) * scale
    late = torch.arange(len(k), device=q.device)[None] > first + torch.arange(q.shape[1], device=q.device)[:, None]
    return torch.softmax(x.masked_fill_(late, -math.inf), -1) @ v


def _exact_append(case, s):
    d, bs, hkv, pool = case["d"], case["bs"], case["hkv"], case["pool"]
    ks, vs = s["kst"].double(), s["vst"].double()
    half = case["rot"] // 2
    cs = s["cos_sin"].double()[s["pos"].long()]
    i = torch.arange(half, device="cuda")
    a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
    turned = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        x = x * (x.square().sum(-1, keepdim=True) / d + EPS).rsqrt() * w.double()
        y = x.clone()
        y[..., a] = x[..., a] * cs[:, None, :half] - x[..., b] * cs[:, None, half:]
        y[..., b] = x[..., b] * cs[:, None, :half] + x[..., a] * cs[:, None, half:]
        turned[name] = y
    kept = s["slots"] >= 0
    r = {"q": turned["q"] * kept[:, None, None]}
    if case["keys"]:
        r["keys"] = turned["k"] * kept[:, None, None]
    slot, blocks = s["slots"][kept], s["blocks"].long()
    for name, new, pooled, scale in (("k", turned["k"], s["kp"], ks), ("v", s["v"].double(), s["vp"], vs)):
        if pool == "fp4":
            full = torch.zeros((pooled.shape[0], hkv, bs, d), dtype=torch.float64, device="cuda")
            full[blocks] = _block64(pooled, pool, blocks, bs, d) * scale
        else:
            full = _e4m3(pooled) if pool == "fp8" else pooled.double()
        full[slot // bs, :, slot % bs] = _store64(pool, new[kept], scale)
        r[name] = full[blocks] if pool == "fp4" else full
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm_rope":
        return _exact_append(case, s)
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    g, starts = hq // hkv, s["starts"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i in range(case["b"]):
        at, n = starts[i], starts[i + 1] - starts[i]
        if n == 0:
            continue
        for h in range(hkv):
            q = s["q"][at:at + n, h * g:(h + 1) * g].double().transpose(0, 1)
            if case["kind"] == "prompt":
                k, v, first = s["k"][at:at + n, h].double(), s["v"][at:at + n, h].double(), 0
            else:
                t, bs = int(s["lens"][i]), case["bs"]
                table = s["tables"][i, : -(-t // bs)]
                k, v = (_block64(p[:, h:h + 1], case["pool"], table, bs, d).reshape(-1, d)[:t] * scale.double()
                        for p, scale in ((s["kp"], s["kst"]), (s["vp"], s["vst"])))
                first = t - n
            out[at:at + n, h * g:(h + 1) * g] = _rows64(q, k, v, first, s["scale"]).transpose(0, 1)
    return {"out": out}
