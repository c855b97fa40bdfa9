"""What a decode step does around and over a 4-bit key/value cache, in plain torch and through the library's calls.

The operators, each measured over the sizes that the workloads of this package have:

  rope     rotary positions on queries and keys: half and interleaved pairs, whole heads or their first `rot` dims
  append   the same rotation with the new keys and values appended to a paged cache: 16-bit, FP8 E4M3 or 4-bit
  write    new keys and values quantised into a 4-bit cache
  decode   attention of one or a few query tokens per sequence over a 4-bit paged cache

A 4-bit cache is uint8 [blocks, KV heads, 8 * D + 64]: a (block, KV head) chunk is 16 token rows of D / 2 bytes (element 2i in the low
nibble of byte i) and then each row's bfloat16 (scale, low); an element is code * scale + low. What is written in 4 bits is read back as
16-bit rows (`pa_gather_cache`), so that a pass returns the values that the codes stand for.

`own` chooses between the plain form and the library (paged_kv_cache_424_b200.binding).
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 16  # tokens per cache block


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token of the small fp16 shape: nothing but latency
        dict(name="rope_one", op="rope", dtype="fp16", tokens=1, heads=8, kv_heads=8, dim=64, rot=64, pairs="interleaved", magnitude=1.0, far=4000),
        # a chunk of prompts on the 8B shape at positions of a long context, the magnitude of a context extended eightfold
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, pairs="half", magnitude=1.2079, far=131072),
        # one decode step of 256 sequences on the 8B shape, a 16-bit cache
        dict(name="append16_step", op="append", cache="16", dtype="bf16", tokens=256, heads=32, kv_heads=8, dim=128, rot=128, pairs="half", magnitude=1.0, far=4096, blocks=4096, padding=0.0),
        # a prompt chunk on the 7B shape into an FP8 cache, half of each head rotated; a few padding tokens
        dict(name="append8_prompt", op="append", cache="fp8", dtype="fp16", tokens=4093, heads=32, kv_heads=32, dim=128, rot=64, pairs="interleaved", magnitude=1.0, far=8192, blocks=512, padding=0.02),
        # a prompt chunk on the 70B shape into a 4-bit cache, read back
        dict(name="append4_prompt", op="append", cache="int4", dtype="bf16", tokens=8192, heads=64, kv_heads=8, dim=128, rot=128, pairs="half", magnitude=1.0, far=32768, blocks=2048, padding=0.0),
        # the new tokens of 64 sequences on the 7B shape, written and read back
        dict(name="write4_step", op="write", dtype="fp16", tokens=64, kv_heads=32, dim=128, blocks=1024, padding=0.0),
        # many ragged prompts at head_dim 64, padded to a captured size
        dict(name="write4_ragged", op="write", dtype="bf16", tokens=20001, kv_heads=8, dim=64, blocks=2048, padding=0.07),
        # the four short sequences of the smallest workload
        dict(name="decode4_tiny", op="decode", dtype="fp16", lens="1,17,33,100", seqs=4, heads=8, kv_heads=8, dim=64, queries=1, window=0),
        # 64 sequences of 128 to 2048 tokens on the 7B shape: a KV head for every query head
        dict(name="decode4_mha7b", op="decode", dtype="fp16", lens="uniform:128:2048:1", seqs=64, heads=32, kv_heads=32, dim=128, queries=1, window=0),
        # continuous batching on the 8B shape
        dict(name="decode4_gqa8b", op="decode", dtype="bf16", lens="lognormal:1024:4096:2", seqs=256, heads=32, kv_heads=8, dim=128, queries=1, window=0),
        # long contexts on the 70B shape
        dict(name="decode4_long70b", op="decode", dtype="bf16", lens="uniform:32768:32768:3", seqs=8, heads=64, kv_heads=8, dim=128, queries=1, window=0),
        # draft tokens verified on the 8B shape: four query tokens per sequence
        dict(name="decode4_spec8b", op="decode", dtype="bf16", lens="lognormal:1024:4096:5", seqs=256, heads=32, kv_heads=8, dim=128, queries=4, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "write", "decode", "decode"))
    dtype, dim = rng.choice(("fp16", "bf16")), rng.choice((64, 128, 128))
    kv = rng.choice((1, 2, 4, 8, 32))
    group = rng.choice((1, 2, 4, 8, 16)) if kv <= 4 else rng.choice((1, 4, 8)) if kv == 8 else 1
    head = dict(op=op, dtype=dtype, heads=kv * group, kv_heads=kv, dim=dim)
    if op == "decode":
        most = rng.choice((700, 4096, 20000, 32768))
        seqs = _log(rng, 1, max(2, min(256, 260000 * 8 // (most * kv))))
        queries = rng.choice([n for n in (1, 1, 2, 3, 4) if n * group <= 16])
        window = rng.choice((0, 0, 0, _log(rng, 16, most)))
        kind = rng.choice(("uniform:%d:%d:%d" % (max(1, most // 16), most, rng.randrange(1 << 20)), "lognormal:%d:%d:%d" % (max(1, most // 4), most, rng.randrange(1 << 20))))
        return dict(head, lens=kind, seqs=seqs, queries=queries, window=window)
    tokens = _log(rng, 1, 8192 * 8 // max(8, kv))
    if op == "write":
        return dict(op=op, dtype=dtype, tokens=tokens, kv_heads=kv, dim=dim, blocks=tokens // BLOCK + _log(rng, 8, 1000), padding=rng.choice((0.0, 0.1)))
    turn = dict(tokens=tokens, rot=rng.choice((dim, dim, dim // 2, dim // 4, 2 * rng.randrange(1, dim // 2))), pairs=rng.choice(("half", "interleaved")),
                magnitude=rng.choice((1.0, 1.1386)), far=_log(rng, 4096, 131072))
    if op == "rope":
        return dict(head, **turn)
    return dict(head, **turn, cache=rng.choice(("16", "fp8", "int4")), blocks=tokens // BLOCK + _log(rng, 8, 1000), padding=rng.choice((0.0, 0.1)))


def lengths(case):
    """The context lengths of a decode case: part of the case, the same for every seed."""
    kind = case["lens"].split(":")
    if len(kind) == 1:
        return [int(n) for n in case["lens"].split(",")]
    rng, low, most = random.Random(int(kind[3])), int(kind[1]), int(kind[2])
    if kind[0] == "uniform":
        return [rng.randint(low, most) for _ in range(case["seqs"])]
    return [min(most, max(case["queries"], round(low * math.exp(rng.gauss(0.0, 1.0))))) for _ in range(case["seqs"])]


def work(case):
    """Each input once, each output once: queries and keys in and out, cache rows written or read, tables, slots and positions."""
    D, Hk = case["dim"], case["kv_heads"]
    if case["op"] == "decode":
        lens = lengths(case)
        reach = [min(n, case["window"] + case["queries"] - 1) if case["window"] else n for n in lens]
        row = 2 * Hk * (D // 2 + 4)
        qo = 2 * 2 * case["seqs"] * case["queries"] * case["heads"] * D
        return {"bytes": sum(reach) * row + sum(4 * -(-n // BLOCK) + 4 for n in reach) + qo, "flops": 4 * sum(reach) * case["queries"] * case["heads"] * D}
    T = case["tokens"]
    kv = 2 * T * Hk * D  # elements of the keys and the values
    if case["op"] == "rope":
        n = T * (case["heads"] + Hk) * D
        return {"bytes": 4 * n + 8 * T, "flops": 3 * n * case["rot"] // D}
    stored = {"16": 2 * D, "fp8": D, "int4": D // 2 + 4}[case.get("cache", "int4")] * 2 * T * Hk
    again = 2 * kv if case.get("cache", "int4") == "int4" else 0  # the rows read back
    if case["op"] == "write":
        return {"bytes": 2 * kv + stored + again + 8 * T, "flops": 3 * kv}
    n = T * case["heads"] * D
    return {"bytes": 4 * n + 2 * kv + stored + again + 16 * T, "flops": 3 * (n + kv // 2) * case["rot"] // D + 2 * kv}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tokens(gen, T, heads, D):
    """Projections of `heads` heads: normal values, a few channels of every head much larger, as keys have them."""
    x = torch.randn((T, heads, D), generator=gen, device="cuda")
    return x * (1.0 + 4.0 * (torch.rand((heads, D), generator=gen, device="cuda") < 0.05))


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    T16, D, Hk = TYPES[case["dtype"]], case["dim"], case["kv_heads"]
    s = dict(case=case)
    if case["op"] == "decode":
        lens = lengths(case)
        S, QL, H = len(lens), case["queries"], case["heads"]
        row = max(1, -(-max(lens) // BLOCK))
        used = sum(-(-n // BLOCK) for n in lens)
        NB = used + 64
        perm = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32)
        tables, at = torch.full((S, row), -1, dtype=torch.int32, device="cuda"), 0
        for i, n in enumerate(lens):
            b = -(-n // BLOCK)
            tables[i, :b] = perm[at:at + b]
            at += b
        for name in ("k_cache", "v_cache"):
            pool = torch.randint(0, 256, (NB, Hk, 8 * D + 64), generator=gen, device="cuda", dtype=torch.uint8)
            scales = 0.3 * torch.exp(torch.randn((NB, Hk, BLOCK), generator=gen, device="cuda") * 0.3).to(torch.bfloat16)
            lows = (scales.float() * (-7.5 + torch.randn((NB, Hk, BLOCK), generator=gen, device="cuda"))).to(torch.bfloat16)
            pool[:, :, 8 * D:] = torch.stack((scales, lows), -1).view(torch.uint8).view(NB, Hk, 64)
            s[name] = pool
        shape = (S, QL, H, D) if QL > 1 or case["window"] else (S, H, D)
        s.update(q=(2.0 * torch.randn(shape, generator=gen, device="cuda")).to(T16), tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 longest=max(lens), scale=1.0 / math.sqrt(D), workspace=torch.empty(_WORKSPACE, dtype=torch.uint8, device="cuda"))
        s["out"] = torch.empty_like(s["q"])
        return s
    T = case["tokens"]
    if case["op"] in ("rope", "append"):
        # one projection's output holds queries, keys and values side by side: the calls read views of it
        H = case["heads"]
        qkv = _tokens(gen, T, H + 2 * Hk, D).to(T16)
        s.update(q=qkv[:, :H], key=qkv[:, H:H + Hk], value=qkv[:, H + Hk:], q_out=torch.zeros((T, H, D), dtype=T16, device="cuda"),
                 k_out=torch.zeros((T, Hk, D), dtype=T16, device="cuda"),
                 positions=torch.randint(0, case["far"], (T,), generator=gen, device="cuda"),
                 inv_freq=torch.exp(torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") * (-math.log(500000.0) / case["rot"])))
        if case["op"] == "rope":
            return s
    else:
        s.update(key=_tokens(gen, T, Hk, D).to(T16), value=_tokens(gen, T, Hk, D).to(T16))
    NB, cache = case["blocks"], case.get("cache", "int4")
    slots = torch.randperm(NB * BLOCK, generator=gen, device="cuda")[:T]
    s["slots"] = torch.where(torch.rand((T,), generator=gen, device="cuda") < case["padding"], torch.full_like(slots, -1), slots)
    shape = (NB, Hk, 8 * D + 64) if cache == "int4" else (NB, Hk, BLOCK, D)
    kind = {"16": T16, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}[cache]
    s.update(k_cache=torch.zeros(shape, dtype=torch.uint8 if cache != "16" else kind, device="cuda").view(kind),
             v_cache=torch.zeros(shape, dtype=torch.uint8 if cache != "16" else kind, device="cuda").view(kind),
             k_scale=0.11 if cache == "fp8" else 1.0, v_scale=0.07 if cache == "fp8" else 1.0)
    if cache == "int4":
        s.update(k_read=torch.zeros((T, Hk, D), dtype=T16, device="cuda"), v_read=torch.zeros((T, Hk, D), dtype=T16, device="cuda"))
    return s


_WORKSPACE = 160 << 20  # bytes kept for partial results: every case's plan fits


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return (_own if own else _plain)(s, s["case"])


def _own(s, case):
    from paged_kv_cache_424_b200 import binding as pa
    if case["op"] == "decode":
        if s["q"].dim() == 4:
            return pa.pa_decode_ext(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"], case["kv_heads"], s["longest"],
                                    q_len=case["queries"], window=case["window"], workspace=s["workspace"])
        return pa.pa_decode_int4(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"], case["kv_heads"], s["longest"], workspace=s["workspace"])
    if case["op"] == "write":
        pa.pa_reshape_and_cache_int4(s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"])
        pa.pa_gather_cache(s["k_read"], s["v_read"], s["k_cache"], s["v_cache"], s["slots"])
        return s["k_read"], s["v_read"]
    turn = dict(interleaved=case["pairs"] == "interleaved", magnitude=case["magnitude"])
    if case["op"] == "rope":
        pa.pa_rope(s["q_out"], s["q"], s["k_out"], s["key"], s["positions"], s["inv_freq"], **turn)
        return s["q_out"], s["k_out"]
    pa.pa_rope_and_cache(s["q_out"], s["q"], s["key"], s["value"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["inv_freq"], **turn,
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
    if case["cache"] != "int4":
        return s["q_out"], s["k_cache"], s["v_cache"]
    pa.pa_gather_cache(s["k_read"], s["v_read"], s["k_cache"], s["v_cache"], s["slots"])
    return s["q_out"], s["k_read"], s["v_read"]


def _rotate(x, positions, inv_freq, case):
    """Pairs (a, b) of a head's first `rot` dims become (a cos - b sin, b cos + a sin); float32, angles in float64."""
    x, rot = x.float(), case["rot"]
    angle = positions.double()[:, None] * inv_freq[None, :]
    cos, sin = ((f(angle) * case["magnitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    if case["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _quantised(x):
    """Rows of float32 -> (codes 0..15, bfloat16 scale and low): low = the smallest element, scale = (largest - low) / 15."""
    low = x.amin(-1).to(torch.bfloat16)
    scale = ((x.amax(-1) - low.float()) / torch.full((), 15.0, device=x.device)).to(torch.bfloat16)
    y = torch.round((x - low.float()[..., None]) / scale.float()[..., None]).clamp(0.0, 15.0)
    return torch.where(scale[..., None] != 0, y, torch.zeros_like(y)).int(), torch.stack((scale, low), -1)


def _put4(pool, x, slots, D):
    """Rows of a 4-bit cache from float32 [n, Hk, D]; padding tokens leave it as it was."""
    live = slots >= 0
    at, x = slots[live], x[live]
    code, ends = _quantised(x)
    pool[:, :, :8 * D].unflatten(2, (BLOCK, D // 2))[at // BLOCK, :, at % BLOCK] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
    pool[:, :, 8 * D:].unflatten(2, (BLOCK, 4))[at // BLOCK, :, at % BLOCK] = ends.view(torch.uint8)


def _values4(codes, ends):
    """Packed codes [..., D / 2] and their rows' (scale, low) as 4 bytes -> float32 [..., D]."""
    ends = ends.contiguous().view(torch.bfloat16).float()
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2) * ends[..., :1] + ends[..., 1:]


def _get4(out, pool, slots, D):
    live = slots >= 0
    at = slots[live]
    codes = pool[:, :, :8 * D].unflatten(2, (BLOCK, D // 2))[at // BLOCK, :, at % BLOCK]
    ends = pool[:, :, 8 * D:].unflatten(2, (BLOCK, 4))[at // BLOCK, :, at % BLOCK]
    out[live] = _values4(codes, ends).to(out.dtype)
    return out


def _put(pool, x, slots, scale):
    live = slots >= 0
    at = slots[live]
    y = x[live] if pool.dtype != torch.float8_e4m3fn else (x[live] / torch.full((), scale, device=x.device)).clamp(-448.0, 448.0)
    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
    raw[at // BLOCK, :, at % BLOCK] = y.to(pool.dtype).view(raw.dtype)


def _plain(s, case):
    D = case["dim"]
    if case["op"] == "decode":
        return _attend(s, case)
    if case["op"] == "write":
        for pool, x in ((s["k_cache"], s["key"]), (s["v_cache"], s["value"])):
            _put4(pool, x.float(), s["slots"], D)
        return _get4(s["k_read"], s["k_cache"], s["slots"], D), _get4(s["v_read"], s["v_cache"], s["slots"], D)
    q, k = (_rotate(s[n], s["positions"], s["inv_freq"], case) for n in ("q", "key"))
    if case["op"] == "rope":
        s["q_out"].copy_(q)
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    live = s["slots"] >= 0
    s["q_out"][live] = q[live].to(s["q_out"].dtype)
    if case["cache"] != "int4":
        _put(s["k_cache"], k, s["slots"], s["k_scale"])
        _put(s["v_cache"], s["value"].float(), s["slots"], s["v_scale"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    _put4(s["k_cache"], k, s["slots"], D)
    _put4(s["v_cache"], s["value"].float(), s["slots"], D)
    return s["q_out"], _get4(s["k_read"], s["k_cache"], s["slots"], D), _get4(s["v_read"], s["v_cache"], s["slots"], D)


def _attend(s, case):
    """Every sequence padded to the longest: gather, scores, masked softmax, weighted sum, in float32."""
    D, Hk, QL = case["dim"], case["kv_heads"], case["queries"]
    q = s["q"].float().reshape(len(s["lens"]), QL, Hk, case["heads"] // Hk, D)
    row = s["tables"].shape[1]
    tables = s["tables"].clamp(min=0).long()

    def cached(pool):
        chunk = pool[tables]  # [S, row, Hk, 8 D + 64]
        x = _values4(chunk[..., :8 * D].unflatten(-1, (BLOCK, D // 2)), chunk[..., 8 * D:].unflatten(-1, (BLOCK, 4)))
        return x.transpose(1, 2).reshape(len(tables), Hk, row * BLOCK, D)

    at = torch.arange(row * BLOCK, device=q.device)
    here = s["lens"][:, None] - QL + torch.arange(QL, device=q.device)[None, :]  # position of each query
    seen = at[None, None, :] <= here[:, :, None]
    if case["window"]:
        seen &= at[None, None, :] > here[:, :, None] - case["window"]
    x = torch.einsum("sqhgd,shtd->sqhgt", q, cached(s["k_cache"])) * s["scale"]
    x = x.masked_fill(~seen[:, :, None, None, :], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3.0e38))
    total = x.sum(-1, keepdim=True)
    o = torch.einsum("sqhgt,shtd->sqhgd", x, cached(s["v_cache"])) / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(o.reshape(s["out"].shape))
    return s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "write": _exact_write, "rope": _exact_rope, "append": _exact_append}[case["op"]](s, case)


def _exact_turn(x, s, case):
    """The rotation as a product of complex numbers."""
    rot, x = case["rot"], x.double()
    turn = torch.polar(torch.full((), case["magnitude"], dtype=torch.float64, device=x.device), s["positions"].double()[:, None] * s["inv_freq"])[:, None, :]
    out = x.clone()
    if case["pairs"] == "half":
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    return out


def _exact_rope(s, case):
    return _exact_turn(s["q"], s, case), _exact_turn(s["key"], s, case)


def _exact_row4(x, slots):
    """Rows as a 4-bit cache holds them: the nearest of a row's sixteen values, found by distance; even codes first, so that they win ties."""
    low = x.amin(-1, keepdim=True).to(torch.bfloat16).double()
    scale = ((x.amax(-1, keepdim=True) - low) / 15.0).to(torch.bfloat16).double()
    out = torch.empty_like(x)
    for i in range(0, len(x), 1024):
        part = slice(i, i + 1024)
        grid = low[part] + scale[part] * torch.tensor([*range(0, 16, 2), *range(1, 16, 2)], dtype=torch.float64, device=x.device)
        best = (x[part][..., None] - grid[..., None, :]).abs().argmin(-1)
        out[part] = grid.gather(-1, best)
    return out * (slots >= 0)[:, None, None]


def _exact_write(s, case):
    return _exact_row4(s["key"].double(), s["slots"]), _exact_row4(s["value"].double(), s["slots"])


def _exact_append(s, case):
    live = s["slots"] >= 0
    q, k, v = _exact_turn(s["q"], s, case) * live[:, None, None], _exact_turn(s["key"], s, case), s["value"].double()
    if case["cache"] == "int4":
        return q, _exact_row4(k, s["slots"]), _exact_row4(v, s["slots"])
    pools = []
    for name, x, scale in (("k_cache", k, s["k_scale"]), ("v_cache", v, s["v_scale"])):
        pool = torch.zeros(s[name].shape, dtype=torch.float64, device=x.device)
        at = s["slots"][live]
        pool[at // BLOCK, :, at % BLOCK] = x[live] / float(np.float32(scale)) if case["cache"] == "fp8" else x[live]
        pools.append(pool)
    return (q, *pools)


def _exact_decode(s, case):
    """Sequence by sequence, over the positions that each query attends to."""
    D, Hk, QL, H = case["dim"], case["kv_heads"], case["queries"], case["heads"]
    q = s["q"].double().reshape(-1, QL, H, D)
    out = torch.zeros_like(q)

    def cached(pool, blocks, n):
        chunk = pool[blocks]
        code = chunk[..., :8 * D].reshape(len(blocks), Hk, BLOCK, D // 2)
        x = torch.empty((len(blocks), Hk, BLOCK, D), dtype=torch.float64, device="cuda")
        for k, c in ((0, code % 16), (1, code // 16)):
            x[..., k::2] = c.double()
        ends = chunk[..., 8 * D:].contiguous().view(torch.bfloat16).double().reshape(len(blocks), Hk, BLOCK, 2)
        return (x * ends[..., :1] + ends[..., 1:]).permute(0, 2, 1, 3).reshape(-1, Hk, D)[:n]

    for i, n in enumerate(lengths(case)):
        blocks = s["tables"][i, :-(-n // BLOCK)].long()
        k, v = cached(s["k_cache"], blocks, n), cached(s["v_cache"], blocks, n)
        for j in range(QL):
            p = n - QL + j
            if p < 0:
                continue
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            x = torch.einsum("hgd,thd->hgt", q[i, j].reshape(Hk, H // Hk, D), k[lo:p + 1]) * s["scale"]
            out[i, j] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v[lo:p + 1]).reshape(H, D)
    return out.reshape(s["out"].shape)
