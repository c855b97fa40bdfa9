"""GPU parity of rotary positions and of the rotating cache write against
plain 64-bit forms (kv4_ref): pair layouts, partial and odd rotated dims,
strides, in place, far positions, the inverse as gradient, every cache type,
padding, the device error word, graphs and streams.
"""
import pytest
import torch

import kv4_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    from paged_kv_cache_424_b200 import build
    build.build()
    from paged_kv_cache_424_b200 import binding
    assert binding.pa_device_error() == 0, "device error word set before the test"
    yield
    assert binding.pa_device_error() == 0, "a kernel flagged a device error"


def pa():
    from paged_kv_cache_424_b200 import binding
    return binding


def gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def rand(g, shape, dtype, k=1.0):
    return (k * torch.randn(shape, generator=g, device="cuda")).to(dtype)


def freqs(R, base=10000.0):
    return pa().pa_rope_frequencies(R, base)[0].cuda()


def check_rope(q, k, pos, f, inter, mag=1.0, inverse=False, what="", **kw):
    qo, ko = (None if x is None else torch.full(x.shape, float("nan"), dtype=x.dtype, device="cuda") for x in (q, k))
    pa().pa_rope(qo, q, ko, k, pos, f, interleaved=inter, magnitude=mag, inverse=inverse, **kw)
    torch.cuda.synchronize()
    for got, x, n in ((qo, q, "q"), (ko, k, "k")):
        if x is not None:
            ref.near(got, ref.rotate(x, pos, f, inter, mag, inverse), ref.rotate_bound(x, f, inter, mag), f"{what} {n}")
    return qo, ko


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (128, 32), (128, 20), (128, 126), (128, 2), (64, 64), (64, 16),
                                 (64, 6), (64, 34)])
def test_layouts_and_rotated_dims(dtype, inter, D, R):
    g = gen(R + D)
    for T, H, Hk in ((1, 8, 8), (5, 7, 1), (33, 32, 8)):
        pos = torch.randint(0, 5000, (T,), generator=g, device="cuda")
        check_rope(rand(g, (T, H, D), dtype), rand(g, (T, Hk, D), dtype), pos, freqs(R), inter, 1.25, what=f"T={T}")


@pytest.mark.parametrize("inter", [False, True])
def test_views_of_a_fused_projection(inter):
    g = gen(3)
    for dtype, D, H, Hk, T in ((torch.bfloat16, 128, 32, 8, 70), (torch.float16, 64, 3, 1, 9)):
        qkv = rand(g, (T, H + 2 * Hk, D), dtype)
        before = qkv.clone()
        pos = torch.randint(0, 9000, (T,), generator=g, device="cuda")
        check_rope(qkv[:, :H], qkv[:, H:H + Hk], pos, freqs(D), inter)
        check_rope(qkv[:, :H], None, pos, freqs(D), inter)
        check_rope(None, qkv[:, H:H + Hk], pos, freqs(D), inter)
        assert torch.equal(qkv, before)


@pytest.mark.parametrize("R", [128, 64, 20])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place(R, inter):
    g = gen(4)
    q, k = rand(g, (40, 16, 128), torch.bfloat16), rand(g, (40, 2, 128), torch.bfloat16)
    pos = torch.randint(0, 4000, (40,), generator=g, device="cuda")
    qo, ko = check_rope(q, k, pos, freqs(R), inter)
    pa().pa_rope(q, q, k, k, pos, freqs(R), interleaved=inter)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_no_tokens_and_empty_tail():
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    pos = torch.zeros(0, dtype=torch.int64, device="cuda")
    pa().pa_rope(q, q, None, None, pos, freqs(64))
    pool = torch.zeros((4, 4, 16, 64), dtype=torch.float16, device="cuda")
    pa().pa_rope_and_cache(q, q, q, q, pool, pool.clone(), pos, pos, freqs(64))
    assert not pool.any()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_products_and_sums_are_rounded_one_by_one(dtype, inter):
    """Bit for bit the fp32 form with every operation rounded (a product fused
    into the sum moves about one fp16 result in 50,000).  Frequencies are powers
    of two and positions small, so that the angles are exact and the sines
    of two fp64 implementations, which agree to about 1e-15, round to one fp32
    number but for about one in 10^7."""
    g = gen(77)
    T, H, D = 512, 64, 128
    q = rand(g, (T, H, D), dtype, 2.0)
    f = torch.ldexp(torch.ones(D // 2, dtype=torch.float64, device="cuda"), -(torch.arange(D // 2, device="cuda") // 8).int())
    pos = torch.arange(T, device="cuda") % 8
    out = torch.empty_like(q)
    pa().pa_rope(out, q, None, None, pos, f, interleaved=inter)
    angle = pos.double()[:, None] * f
    co, si = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = q.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :D // 2], x[..., D // 2:])
    ac, bs, bc, as_ = a * co, b * si, b * co, a * si
    turned = (ac - bs, bc + as_)
    want = (torch.stack(turned, -1).flatten(-2) if inter else torch.cat(turned, -1)).to(dtype)
    assert torch.equal(out, want)


def test_positions_far_away():
    """fp32 angles would be off by 0.06 rad at 10^6; fp64 ones are off by less
    than 2^-52 * 10^6 * 3 = 7e-10 there, far below fp32's half step.  At 2^31
    the angle's own error, 2^31 * 3 * 2^-53 = 7e-7 rad, is what the bound adds."""
    g = gen(5)
    f = freqs(128, 500000.0)
    pos = torch.tensor([0, 1, 10 ** 6, 131071, 2 ** 24 + 1, -5], device="cuda")
    for inter in (False, True):
        q = rand(g, (6, 4, 128), torch.float16)
        check_rope(q, None, pos, f, inter)
        far = torch.full((6,), 2 ** 31, device="cuda")
        out = torch.empty_like(q)
        pa().pa_rope(out, q, None, None, far, f, interleaved=inter)
        torch.cuda.synchronize()
        slack = ref.rotate_bound(q, f, inter) * (1 + 7e-7 / (3 * 2.0 ** -24))
        ref.near(out, ref.rotate(q, far, f, inter), slack, "2^31")


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(inter):
    """<g, rotate(x)> has the gradient rotate_inverse(g): against the formula,
    and against central differences of the 64-bit rotation (a linear map:
    differences with step 1 are exact up to rounding)."""
    g = gen(6)
    T, H, D, R, m = 6, 3, 64, 48, 1.3
    f = freqs(R)
    pos = torch.randint(0, 3000, (T,), generator=g, device="cuda")
    x, dy = rand(g, (T, H, D), torch.float16), rand(g, (T, H, D), torch.float16)
    dx, _ = check_rope(dy, None, pos, f, inter, m, inverse=True)
    probe = torch.randint(0, T * H * D, (24,), generator=g, device="cuda").tolist()
    for i in probe:
        e = torch.zeros(T * H * D, dtype=torch.float64, device="cuda")
        e[i] = 1.0
        e = e.view(T, H, D)
        diff = ((ref.rotate(x.double() + e, pos, f, inter, m) - ref.rotate(x.double() - e, pos, f, inter, m)) / 2 *
                dy.double()).sum()
        # the kernel's rounding to fp16, and the differences' own rounding
        assert abs(float(diff) - float(dx.view(-1)[i])) <= 2.0 ** -11 * abs(float(diff)) + 1e-6
    # there and back: R^T R = m^2
    y = torch.empty_like(x)
    pa().pa_rope(y, x, None, None, pos, f, interleaved=inter, magnitude=m)
    back = torch.empty_like(x)
    pa().pa_rope(back, y, None, None, pos, f, interleaved=inter, magnitude=1 / m, inverse=True)
    # y is off by 2^-11 |y|, |y| <= m (|a| + |b|) <= 1.3 * 2 * max|x|; back's own rounding on top
    tol = 2.0 ** -10 * 2.1 * float(x.abs().max()) * 2
    assert float((back.double() - x.double()).abs().max()) <= tol


# ---------------------------------------------------------------------------
# the rotating cache write
# ---------------------------------------------------------------------------
def pools_of(kind, NB, Hk, D, dtype, g):
    """Pools of random bytes that are no NaN (so that equality shows every byte that changed)."""
    if kind == "int4":
        return [ref.random_pool(g, NB, Hk, D) for _ in range(2)]
    if kind == "fp8":
        return [torch.randint(0, 0x70, (NB, Hk, 16, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    return [rand(g, (NB, Hk, 16, D), dtype) for _ in range(2)]


def check_cache_row(kind, pool, slots, want, slack, scale, what):
    """Rows of the pool at `slots` (all >= 0) hold `want` (float64, known to within slack) in the pool's type."""
    b, o = slots // 16, slots % 16
    if kind == "16":
        return ref.near(pool[b, :, o], want, slack, what)
    if kind == "fp8":
        got = pool.view(torch.float8_e4m3fn)[b, :, o].double() * scale
        bound = slack + (2.0 ** -4 + 2.0 ** -23) * (want.abs() + slack) + 2.0 ** -10 * scale
        over = want.abs() > 448 * scale
        assert bool((((got - want).abs() <= bound) | (over & (got.abs() == 448 * scale))).all()), what
        return
    # 4-bit: low and scale are the smallest element's and the step's bf16
    # roundings; then every element within half a step, or the range's rounding
    D = want.shape[-1]
    codes, tail = ref.pool_views(pool)
    e = tail[b, :, o].contiguous().view(torch.bfloat16).double().reshape(*want.shape[:2], 2)
    step, low = e[..., 0], e[..., 1]
    s = slack.amax(-1)
    lo, hi = want.amin(-1), want.amax(-1)
    assert bool(((low - lo).abs() <= 2.0 ** -8 * (lo.abs() + s) + s).all()), what + ": low"
    want_step = (hi - low) / 15
    assert bool(((step - want_step).abs() <= (2.0 ** -8 + 2.0 ** -22) * want_step.abs() + s / 7).all()), what + ": scale"
    got = ref.values(pool)[b, :, o]
    # inside [low, low + 15 step]: half a step; outside it: clamped to the end
    # (the end's own rounding); fp32 arithmetic of (x - low) / step: 4 half
    # steps of at most 16 steps
    end = torch.minimum(torch.maximum(want, low[..., None]), (low + 15 * step)[..., None])
    bound = 0.5 * step[..., None].abs() + slack + 64 * 2.0 ** -24 * step[..., None].abs() + 2.0 ** -23 * low.abs()[..., None]
    assert bool(((got - end).abs() <= bound).all()), what + ": codes"
    assert got.shape[-1] == D


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["16", "fp8", "int4"])
@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (128, 64, True), (64, 64, True), (64, 20, False)])
def test_rope_and_cache(dtype, kind, D, R, inter):
    g = gen(D + R)
    f = freqs(R)
    for T, H, Hk, NB in ((1, 8, 8, 2), (67, 8, 2, 9), (300, 32, 8, 40), (40, 16, 1, 5)):
        qkv = rand(g, (T, H + 2 * Hk, D), dtype, 2.0)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
        slots = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.1, torch.full_like(slots, -1), slots)
        pos = torch.randint(0, 20000, (T,), generator=g, device="cuda")
        kc, vc = pools_of(kind, NB, Hk, D, dtype, g)
        kb, vb = kc.clone(), vc.clone()
        qo = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
        ks, vs = (float(torch.tensor(x)) for x in ((0.05, 0.031) if kind == "fp8" else (1.0, 1.0)))
        pa().pa_rope_and_cache(qo, q, k, v, kc, vc, slots, pos, f, interleaved=inter, magnitude=1.1, k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        live = slots >= 0
        at = slots[live]
        assert bool((qo[~live] == 7.0).all()), "a padding token's query row was written"
        ref.near(qo[live], ref.rotate(q, pos, f, inter, 1.1)[live], ref.rotate_bound(q, f, inter, 1.1)[live], "q")
        check_cache_row(kind, kc, at, ref.rotate(k, pos, f, inter, 1.1)[live], ref.rotate_bound(k, f, inter, 1.1)[live], ks, "K")
        check_cache_row(kind, vc, at, v.double()[live], torch.zeros_like(v.double()[live]), vs, "V")
        # the queries left out: the cache is the same, and everything else is as it was
        kc2, vc2 = kb.clone(), vb.clone()
        pa().pa_rope_and_cache(None, None, k, v, kc2, vc2, slots, pos, f, interleaved=inter, magnitude=1.1, k_scale=ks, v_scale=vs)
        assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
        for now, was in ((kc, kb), (vc, vb)):
            rows = ref.pool_views if kind == "int4" else (lambda x: (x,))
            for a, b in zip(rows(now), rows(was)):
                a, b = a.clone(), b.clone()
                a[at // 16, :, at % 16] = 0
                b[at // 16, :, at % 16] = 0
                assert torch.equal(a, b), "bytes outside the written rows changed"


@pytest.mark.parametrize("kind", ["16", "fp8", "int4"])
def test_value_write_equals_the_unrotated_write(kind):
    """The value half, and the key half at position 0, are bit for bit what the plain cache writes give."""
    g = gen(8)
    T, Hk, D, NB = 90, 4, 128, 8
    k, v = rand(g, (T, Hk, D), torch.bfloat16), rand(g, (T, Hk, D), torch.bfloat16)
    slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
    a, b = pools_of(kind, NB, Hk, D, torch.bfloat16, g)
    c, d = a.clone(), b.clone()
    ks, vs = (0.07, 0.05) if kind == "fp8" else (1.0, 1.0)
    pa().pa_rope_and_cache(None, None, k, v, a, b, slots, torch.zeros_like(slots), freqs(128), k_scale=ks, v_scale=vs)
    if kind == "16":
        pa().pa_reshape_and_cache(k, v, c, d, slots)
    elif kind == "fp8":
        pa().pa_reshape_and_cache_fp8(k, v, c, d, slots, ks, vs)
    else:
        pa().pa_reshape_and_cache_int4(k, v, c, d, slots)
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1.0, 0.0123, 3.7, 1e-30, 3e-38, 1e30, 1.9999999, 2.0 ** -90])
def test_fp8_codes_of_every_16bit_value(dtype, scale):
    """The value half quantises every 16-bit pattern as pa_reshape_and_cache_fp8
    does (a correctly rounded quotient, whichever way it is formed), NaN as NaN."""
    p = pa()
    v = torch.arange(65536, device="cuda").to(torch.int16).view(dtype).view(256, 2, 128)
    pools = [torch.zeros((16, 2, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(4)]
    slots, pos = torch.arange(256, device="cuda"), torch.zeros(256, dtype=torch.int64, device="cuda")
    k = torch.zeros_like(v)
    s = float(torch.tensor(scale, dtype=torch.float32))
    p.pa_rope_and_cache(None, None, k, v, pools[0], pools[1], slots, pos, freqs(128), k_scale=1.0, v_scale=s)
    p.pa_reshape_and_cache_fp8(k, v, pools[2], pools[3], slots, 1.0, s)
    torch.cuda.synchronize()
    nan = (pools[3] & 0x7F) == 0x7F
    assert torch.equal(nan, (pools[1] & 0x7F) == 0x7F) and torch.equal(pools[1][~nan], pools[3][~nan])


@pytest.mark.parametrize("kind", ["none", "16", "int4"])
@pytest.mark.parametrize("H,Hk,D,R,inter", [(1, 1, 64, 64, False), (3, 1, 128, 64, True), (32, 8, 128, 20, False), (32, 8, 128, 128, False)])
def test_many_tokens(kind, H, Hk, D, R, inter):
    """More tokens than CTAs: each walks over several, padding among them."""
    p = pa()
    g = gen(H + D)
    T, NB = 3001, 200
    f = freqs(R)
    qkv = rand(g, (T, H + 2 * Hk, D), torch.bfloat16)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    pos = torch.randint(0, 30000, (T,), generator=g, device="cuda")
    if kind == "none":
        check_rope(q, k, pos, f, inter)
        return
    slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
    slots = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.4, torch.full_like(slots, -1), slots)
    kc, vc = pools_of(kind, NB, Hk, D, torch.bfloat16, g)
    qo = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    p.pa_rope_and_cache(qo, q, k, v, kc, vc, slots, pos, f, interleaved=inter)
    torch.cuda.synchronize()
    live = slots >= 0
    at = slots[live]
    assert bool((qo[~live] == 7.0).all())
    ref.near(qo[live], ref.rotate(q, pos, f, inter)[live], ref.rotate_bound(q, f, inter)[live], "q")
    check_cache_row(kind, kc, at, ref.rotate(k, pos, f, inter)[live], ref.rotate_bound(k, f, inter)[live], 1.0, "K")
    check_cache_row(kind, vc, at, v.double()[live], torch.zeros_like(v.double()[live]), 1.0, "V")


def test_slot_past_the_pool_is_flagged_and_skipped():
    g = gen(9)
    p = pa()
    k = rand(g, (5, 2, 64), torch.float16)
    for kind in ("16", "int4"):
        kc, vc = pools_of(kind, 3, 2, 64, torch.float16, g)
        kb, vb = kc.clone(), vc.clone()
        slots = torch.tensor([48, 1 << 40, -1, -(1 << 50), 48], device="cuda")
        q, pos = torch.full_like(k, 3.0), torch.arange(5, device="cuda")
        p.pa_rope_and_cache(q, k, k, k, kc, vc, slots, pos, freqs(64))
        assert p.pa_device_error() == 4
        assert torch.equal(kc, kb) and torch.equal(vc, vb)
        assert bool((q[2:4] == 3.0).all())
        ref.near(q[[0, 1, 4]], ref.rotate(k, pos, freqs(64), False)[[0, 1, 4]],
                 ref.rotate_bound(k, freqs(64), False)[[0, 1, 4]], "q of a flagged slot")


def test_infinities_and_nan_stay_in_their_pairs():
    g = gen(10)
    x = rand(g, (2, 3, 64), torch.float16)
    clean = torch.empty_like(x)
    pos, f = torch.tensor([3, 4000], device="cuda"), freqs(32)
    pa().pa_rope(clean, x, None, None, pos, f)
    x[0, 1, 5] = float("nan")
    x[1, 2, 40] = float("inf")
    out = torch.empty_like(x)
    pa().pa_rope(out, x, None, None, pos, f)
    torch.cuda.synchronize()
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1, 5] = hit[0, 1, 21] = hit[1, 2, 40] = True
    assert bool(out[0, 1, [5, 21]].isnan().all()) and bool(out[1, 2, 40].isinf())
    assert torch.equal(out[~hit], clean[~hit])


def test_graph_and_other_stream():
    """Captured once and replayed on changed inputs; and on a stream that is not the current one."""
    g = gen(11)
    p = pa()
    T, H, Hk, D, NB = 16, 8, 2, 128, 4
    qkv = rand(g, (T, H + 2 * Hk, D), torch.bfloat16)
    kc, vc = (torch.zeros(p.int4_cache_shape(NB, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots, pos, f = torch.arange(T, device="cuda"), torch.arange(T, device="cuda"), freqs(D)
    qo = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: p.pa_rope_and_cache(qo, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], kc, vc, slots, pos, f, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in (1, 2):
        qkv.copy_(rand(g, qkv.shape, torch.bfloat16))
        pos.add_(17 * step)
        slots.copy_((slots + 5) % (NB * 16))
        graph.replay()
        torch.cuda.synchronize()
        ref.near(qo, ref.rotate(qkv[:, :H], pos, f, False), ref.rotate_bound(qkv[:, :H], f, False), "replay")
    side = torch.cuda.Stream()
    want_q, want_k = qo.clone(), kc.clone()
    qo.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(qo, want_q) and torch.equal(kc, want_k)


@pytest.mark.parametrize("inter,R", [(False, 128), (True, 128), (False, 20)])
def test_keys_alone_and_both_in_place(inter, R):
    """Keys without queries (one head, many heads, many tokens), and queries and keys both in place."""
    g = gen(78)
    f = freqs(R)
    for T, H, Hk in ((1, 1, 1), (3000, 8, 1), (17, 32, 32)):
        q, k = rand(g, (T, H, 128), torch.bfloat16), rand(g, (T, Hk, 128), torch.bfloat16)
        pos = torch.randint(0, 9000, (T,), generator=g, device="cuda")
        _, alone = check_rope(None, k, pos, f, inter, what="keys alone")
        qo, ko = check_rope(q, k, pos, f, inter, what="both")
        assert torch.equal(ko, alone)
        pa().pa_rope(q, q, k, k, pos, f, interleaved=inter)
        assert torch.equal(q, qo) and torch.equal(k, ko)
