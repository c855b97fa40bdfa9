"""Rotary positions, 4-bit caches and read-back: frequencies against their
formulas, plans, and refusals on the host (no GPU: every call returns before
anything is enqueued; the refusals run in a child process that sees none)."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_424_b200 import build
    build.build()
    from paged_kv_cache_424_b200 import binding
    return binding


def plain(R, base):
    return [base ** (-2.0 * i / R) for i in range(R // 2)]


def close(got, want):
    assert got.numel() == len(want)
    for a, b in zip(got.tolist(), want):
        assert abs(a - b) <= 1e-14 * abs(b)


@pytest.mark.parametrize("R,base", [(2, 10000.0), (20, 10000.0), (64, 500000.0), (128, 1e6)])
def test_frequencies_plain_and_linear(lib, R, base):
    f, m = lib.pa_rope_frequencies(R, base)
    close(f, plain(R, base))
    assert m == 1.0
    f, m = lib.pa_rope_frequencies(R, base, "linear", factor=4.0)
    close(f, [x / 4.0 for x in plain(R, base)])
    assert m == 1.0


def test_frequencies_ntk(lib):
    R, base, k = 128, 10000.0, 8.0
    f, _ = lib.pa_rope_frequencies(R, base, "ntk", factor=k)
    p = plain(R, base)
    assert f[0] == 1.0                                    # the fastest pair unchanged
    assert abs(float(f[-1]) - p[-1] / k) <= 1e-13 * p[-1]  # the slowest one as interpolated
    assert all(a <= b for a, b in zip(f.tolist(), p))


def test_frequencies_bands(lib):
    R, base, k, C, lo, hi = 128, 500000.0, 8.0, 8192.0, 1.0, 4.0
    f, m = lib.pa_rope_frequencies(R, base, "bands", factor=k, original_context=C, low_freq_factor=lo,
                                   high_freq_factor=hi)
    want = []
    for x in plain(R, base):
        w = 2 * math.pi / x
        if w < C / hi:
            want.append(x)
        elif w > C / lo:
            want.append(x / k)
        else:
            t = (C / w - lo) / (hi - lo)
            want.append((1 - t) * x / k + t * x)
    close(f, want)
    assert m == 1.0


def test_frequencies_yarn(lib):
    R, base, k, C, fast, slow = 128, 10000.0, 16.0, 4096.0, 32.0, 1.0
    f, m = lib.pa_rope_frequencies(R, base, "yarn", factor=k, original_context=C, beta_fast=fast, beta_slow=slow)
    dim = lambda turns: R * math.log(C / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    a, b = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), R - 1)
    want = []
    for i, x in enumerate(plain(R, base)):
        r = min(max((i - a) / (b - a), 0.0), 1.0)
        want.append(r * x / k + (1 - r) * x)
    close(f, want)
    assert abs(m - (0.1 * math.log(k) + 1.0)) < 1e-15
    assert lib.pa_rope_frequencies(R, base, "yarn", factor=1.0, original_context=C)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="ntk", rotary_dim=2, factor=2.0),
                                dict(scaling="bands", factor=2.0), dict(scaling="yarn", factor=2.0),
                                dict(scaling="bands", factor=2.0, original_context=100.0, low_freq_factor=4.0),
                                dict(scaling="yarn", factor=2.0, original_context=100.0, beta_slow=40.0),
                                dict(scaling="linear", factor=float("inf"))])
def test_frequencies_refused(lib, kw):
    with pytest.raises(lib.PagedAttentionError) as e:
        lib.pa_rope_frequencies(**{"rotary_dim": 64, **kw})
    assert e.value.status == -3
    with pytest.raises(ValueError):
        lib.pa_rope_frequencies(64, scaling="no such thing")


def test_int4_shapes(lib):
    assert lib.int4_cache_shape(5, 3, 128) == (5, 3, 1088)
    assert lib.int4_cache_shape(5, 3, 64) == (5, 3, 576)
    pool = torch.zeros(lib.int4_cache_shape(5, 3, 64), dtype=torch.uint8)
    d = lib.cache_dims(pool, torch.bfloat16)
    assert (d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim, d.dtype, d.kv_dtype) == (5, 3, 16, 64, 1, 3)
    with pytest.raises(ValueError):
        lib.cache_dims(torch.zeros((5, 3, 577), dtype=torch.uint8), torch.float16)


def test_int4_plan_is_consistent(lib):
    """The workspace is zero exactly for one partition; with partitions of a
    given size it holds an fp32 row and an lse for every (query row,
    partition); automatic ones take a workspace that does not grow with the
    batch's contexts."""
    import random
    rng = random.Random(5)
    for _ in range(300):
        hk, g, D = rng.choice((1, 2, 8, 32)), rng.choice((1, 2, 4, 8, 16)), rng.choice((64, 128))
        mb = rng.randint(1, 4096)
        S, P = rng.randint(1, 600), rng.choice((0, 0, 16, 256, 4096))
        d = lib.make_dims(S, hk * g, hk, D, 16, mb, 1000, lib.PA_F16, lib.PA_INT4)
        n = rng.randint(0, mb * 16)
        parts, ws = lib.pa_decode_num_partitions(d, n, P), lib.pa_decode_workspace_size(d, n, P)
        assert parts >= 1
        rows = S * hk * g * parts
        assert (ws == 0) == (parts == 1)
        if not P:
            assert ws <= 40 << 20
        else:
            assert parts == 1 or ws >= rows * D * 4 + rows * 4
            assert parts == max(1, -(-(-(-n // 16)) // (P // 16)))


REFUSALS = r"""
import ctypes, sys
sys.path.insert(0, %(root)r)
from paged_kv_cache_424_b200 import binding as b
L = b.LIB
f = ctypes.c_float
p = ctypes.c_void_p(0x10000)
odd = ctypes.c_void_p(0x10008)
def dims(**kw):
    base = dict(num_seqs=4, num_heads=32, num_kv_heads=8, head_dim=128, block_size=16, max_blocks_per_seq=256,
                num_blocks=1024, dtype=b.PA_BF16, kv_dtype=b.PA_INT4)
    base.update(kw)
    return b.pa_dims(**base)
R = ctypes.byref

# decode over 4-bit caches
def dec(d, ptrs=[p] * 6, nkv=8, maxlen=100, part=0, ws=None, wsb=0, fn=L.pa_decode_int4):
    out, q, k, v, bt, cl = ptrs
    return fn(out, q, k, v, bt, cl, f(0.1), nkv, R(d), maxlen, part, ws, wsb, None)
i4 = dims()
assert dec(dims(kv_dtype=0)) == -2 and dec(dims(kv_dtype=b.PA_FP8_E4M3)) == -2
assert dec(i4, fn=L.pa_decode) == -2 and "pa_decode_int4" in b.pa_last_error()
assert L.pa_decode_fp8(p, p, p, p, p, p, f(.1), f(1), f(1), 8, R(i4), 100, 0, None, 0, None) == -2
assert L.pa_decode_noalloc(p, p, p, p, p, p, f(.1), 8, R(i4), 100, 0, None) == -2
assert dec(dims(kv_dtype=4)) == -2
assert dec(dims(head_dim=96)) == -4 and dec(dims(block_size=32)) == -4 and dec(dims(num_heads=24)) == -4
assert dec(i4, nkv=4) == -3 and dec(i4, maxlen=5000) == -3 and dec(i4, part=24) == -3
for k in (0, 1, 2, 3, 5):
    assert dec(i4, ptrs=[p] * k + [None] + [p] * (5 - k)) == -1
for k in range(4):
    assert dec(i4, ptrs=[p] * k + [odd] + [p] * (5 - k)) == -7
assert dec(i4, maxlen=4096, part=16) == -5
assert dec(dims(num_seqs=0), ptrs=[None] * 6) == 0
O = b.pa_decode_opts
def ext(d, o):
    return L.pa_decode_ext(p, p, p, p, p, p, f(.1), 8, R(d), R(o), 4096, 16, None, 0, None)
assert ext(i4, O(1, 0, 1.0, 1.0)) == -5 and ext(i4, O(5, 0, 1.0, 1.0)) == -4 and ext(i4, O(1, -1, 1.0, 1.0)) == -3
assert ext(i4, O(1, 0, 0.0, 1.0)) == -3

# 4-bit write
def w4(d, key=p, val=p, kc=p, vc=p, sl=p, n=4):
    return L.pa_reshape_and_cache_int4(key, val, kc, vc, sl, n, R(d), None)
assert w4(dims(kv_dtype=0)) == -2 and w4(dims(kv_dtype=2)) == -2
assert L.pa_reshape_and_cache(p, p, p, p, p, 4, R(i4), None) == -2
assert "pa_reshape_and_cache_int4" in b.pa_last_error()
assert L.pa_reshape_and_cache_fp8(p, p, p, p, p, 4, R(i4), f(1), f(1), None) == -2
assert w4(i4, n=-1) == -3 and w4(i4, n=0, key=None) == 0 and w4(dims(num_blocks=0)) == -3
for a in ("key", "val", "kc", "vc", "sl"):
    assert w4(i4, **{a: None}) == -1
for a in ("key", "val", "kc", "vc"):
    assert w4(i4, **{a: odd}) == -7

# read-back
def ga(d, key=p, val=p, kc=p, vc=p, sl=p, n=4, ks=1.0, vs=1.0):
    return L.pa_gather_cache(key, val, kc, vc, sl, n, R(d), f(ks), f(vs), None)
for kv in (0, 1, 2, 3):
    d = dims(kv_dtype=kv)
    assert ga(d, n=-1) == -3 and ga(d, n=0, key=None) == 0
    for a in ("key", "val", "kc", "vc", "sl"):
        assert ga(d, **{a: None}) == -1
    for a in ("key", "val", "kc", "vc"):
        assert ga(d, **{a: odd}) == -7
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert ga(d, ks=s) == -3 and ga(d, vs=s) == -3
assert ga(dims(kv_dtype=0), ks=0.5) == -3
assert ga(dims(kv_dtype=0, dtype=1, head_dim=80)) == -4

# rotation
D = 128
far = lambda k: ctypes.c_void_p(0x100000 * k)
opts = lambda **kw: b.pa_rope_opts(**{**dict(inv_freq=0x10000, rotary_dim=128, interleaved=0, inverse=0, magnitude=1.0), **kw})
def rope(d=dims(kv_dtype=0), o=opts(), qo=far(1), q=far(2), ko=far(3), k=far(4), pos=p, n=4, qs=32 * D, ks=8 * D):
    return L.pa_rope(qo, q, ko, k, pos, n, R(d), R(o) if o is not None else None, qs, ks, None)
assert rope(o=None) == -1 and rope(n=-1) == -3 and rope(n=0) == 0
for o, want in ((dict(rotary_dim=0), -3), (dict(rotary_dim=7), -3), (dict(rotary_dim=130), -3), (dict(interleaved=2), -3),
                (dict(inverse=-1), -3), (dict(magnitude=float("inf")), -3), (dict(magnitude=float("nan")), -3),
                (dict(inv_freq=None), -1)):
    assert rope(o=opts(**o)) == want, o
assert rope(q=None) == -1 and rope(qo=None) == -1 and rope(k=None) == -1 and rope(pos=None) == -1
assert rope(q=None, qo=None, k=None, ko=None) == -1
assert rope(qs=32 * D - 8) == -3 and rope(qs=32 * D + 4) == -3 and rope(ks=0) == -3 and rope(ks=-8 * D) == -3
assert rope(d=dims(kv_dtype=0, num_heads=0)) == -3 and rope(d=dims(kv_dtype=0, num_kv_heads=0)) == -3
assert rope(d=dims(kv_dtype=0, dtype=5)) == -2 and rope(d=dims(kv_dtype=0, head_dim=256)) == -4
for a in ("q", "qo", "k", "ko"):
    assert rope(**{a: odd}) == -7
# overlaps: a shifted output, a strided input in place, one output in the other, an output in the other input
assert rope(qo=ctypes.c_void_p(0x200000 + 256), n=4) == -3
assert rope(qo=far(2), qs=48 * D) == -3
assert rope(ko=ctypes.c_void_p(0x100000 + 1024)) == -3
assert rope(ko=far(2)) == -3 and rope(qo=far(4)) == -3
# rotation + cache write
def rc(d=i4, o=opts(), qo=far(1), q=far(2), k=far(3), v=far(4), kc=far(5), vc=far(6), sl=p, pos=p, n=4, qs=32 * D,
       ks=8 * D, vs=8 * D, a=1.0, c=1.0):
    return L.pa_rope_and_cache(qo, q, k, v, kc, vc, sl, pos, n, R(d), R(o) if o is not None else None, qs, ks, vs, f(a),
                               f(c), None)
assert rc(o=None) == -1 and rc(n=-1) == -3 and rc(n=0) == 0
for name in ("q", "qo", "k", "v", "kc", "vc", "sl", "pos"):
    assert rc(**{name: None}) == -1, name
for name in ("q", "qo", "k", "v", "kc", "vc"):
    assert rc(**{name: odd}) == -7, name
assert rc(o=opts(rotary_dim=200)) == -3 and rc(vs=8) == -3 and rc(ks=8 * D + 2) == -3
assert rc(a=0.5) == -3 and rc(d=dims(kv_dtype=0), c=2.0) == -3 and rc(d=dims(kv_dtype=2), a=0.0) == -3
assert rc(d=dims(kv_dtype=2), c=float("nan")) == -3
assert rc(qo=far(3)) == -3 and rc(qo=far(4)) == -3 and rc(d=dims(kv_dtype=9)) == -2 and rc(d=dims(num_heads=0)) == -3
assert rc(d=dims(block_size=8)) == -4
print("refusals ok")
"""


def test_refusals(lib):
    r = subprocess.run([sys.executable, "-c", REFUSALS % {"root": ROOT}], env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refusals ok" in r.stdout, r.stdout + r.stderr


def test_binding_refuses_host_tensors(lib):
    """Tensors that the kernels could not address never reach them."""
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    pool = torch.zeros(lib.int4_cache_shape(2, 4, 64), dtype=torch.uint8)
    slots = torch.zeros(2, dtype=torch.int64)
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        lib.pa_reshape_and_cache_int4(x, x, pool, pool, slots)
    with pytest.raises(ValueError):
        lib.pa_gather_cache(x, x, pool, pool, slots)
    with pytest.raises(ValueError):
        lib.pa_rope(x, x, None, None, slots, f)
    with pytest.raises(ValueError):
        lib.pa_rope_and_cache(None, None, x, x, pool, pool, slots, slots, f)
    with pytest.raises(ValueError):
        lib.pa_decode_int4(x, x, pool, pool, slots.int()[None], slots.int(), 0.1, 4, 16)
