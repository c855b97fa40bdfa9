"""GPU parity of 4-bit caches: the quantising write and the read-back bit for
bit against the written rule, attention against a 64-bit form within derived
bounds (kv4_ref.attend), block copies, a decode step with its rotation, graphs
and streams.
"""
import numpy as np
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


def same_nan(a, b):
    """Equal bit for bit, a NaN as good as another."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


# ---------------------------------------------------------------------------
# write and read-back
# ---------------------------------------------------------------------------
def edge_rows(D, dtype):
    """Rows where the rule has its edges: constant, zero, one outlier, tiny,
    huge, infinite, NaN, ties, a range that overflows fp32 in bf16."""
    g = gen(1)
    big = 6e4 if dtype == torch.float16 else 3e38
    rows = [torch.zeros(D), -torch.zeros(D), torch.full((D,), 1.003), torch.full((D,), -0.999), torch.full((D,), big),
            torch.arange(D).float() / 16, torch.arange(D).float() % 31 / 2, torch.linspace(-1, 1, D),
            torch.full((D,), 6e-8 if dtype == torch.float16 else 1e-39), torch.linspace(0, 3e-7 if dtype == torch.float16 else 3e-39, D),
            torch.where(torch.arange(D) % 2 == 0, big, -big), torch.where(torch.arange(D) == 3, float("inf"), 1.0),
            torch.where(torch.arange(D) == 9, -float("inf"), 1.0), torch.where(torch.arange(D) == D - 1, float("nan"), 1.0),
            torch.where(torch.arange(D) == 0, 100.0, 0.01), torch.full((D,), float("nan"))]
    more = rand(g, (48, D), torch.float32) * torch.exp(3 * torch.randn((48, 1), generator=g, device="cuda"))
    return torch.cat((torch.stack(rows).cuda(), more)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,Hk", [(64, 1), (64, 8), (128, 1), (128, 8)])
def test_write_bit_for_bit(dtype, D, Hk):
    p = pa()
    rows = edge_rows(D, dtype)
    T = rows.shape[0] // Hk
    key = rows[:T * Hk].view(T, Hk, D).contiguous()
    val = key.flip(0).contiguous()
    g = gen(2)
    NB = T // 16 + 3
    slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
    slots[T // 2] = -1
    kc, vc = (torch.randint(0, 256, p.int4_cache_shape(NB, Hk, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    ek, ev = kc.clone(), vc.clone()
    p.pa_reshape_and_cache_int4(key, val, kc, vc, slots)
    torch.cuda.synchronize()
    for got, want, x in ((kc, ek, key), (vc, ev, val)):
        codes, ends = ref.quantise(x)
        # a NaN's bits are not defined: rows whose ends are NaN are compared as such
        ref.put_rows(want, codes, ends, slots)
        gr, gt = ref.pool_views(got)
        wr, wt = ref.pool_views(want)
        assert torch.equal(gr, wr)
        ge, we = (t.contiguous().view(torch.bfloat16).float() for t in (gt, wt))
        assert same_nan(ge, we)
    # and back: code * scale + low in fp32, rounded once; rows of negative slots stay
    for ks, vs in ((1.0, 1.0), (0.37, 2.5)):
        a, b = torch.full_like(key, 5.0), torch.full_like(key, 5.0)
        p.pa_gather_cache(a, b, kc, vc, slots, ks, vs)
        torch.cuda.synchronize()
        live = slots >= 0
        for got, pool, s in ((a, kc, ks), (b, vc, vs)):
            rows32 = (ref.values(pool, torch.float32) * torch.tensor(s, device="cuda"))[slots[live] // 16, :, slots[live] % 16]
            assert same_nan(got[live], rows32.to(dtype))
            assert bool((got[~live] == 5.0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_gather_16bit_and_fp8(dtype, D):
    """The 16-bit read-back is a copy (NaN payloads included); every E4M3 code widens exactly."""
    p = pa()
    g = gen(3)
    NB, Hk, T = 6, 3, 200
    slots = torch.randint(-20, NB * 16, (T,), generator=g, device="cuda")      # repeated and negative slots
    live = slots >= 0
    at = slots[live]
    raw = torch.randint(-32768, 32768, (2, NB, Hk, 16, D), generator=g, device="cuda", dtype=torch.int16)
    kc, vc = raw[0].view(dtype), raw[1].view(dtype)
    a = torch.zeros((T, Hk, D), dtype=dtype, device="cuda")
    b = torch.zeros_like(a)
    p.pa_gather_cache(a, b, kc, vc, slots)
    torch.cuda.synchronize()
    for got, pool in ((a, raw[0]), (b, raw[1])):
        assert torch.equal(got.view(torch.int16)[live], pool[at // 16, :, at % 16])
        assert not got.view(torch.int16)[~live].any()
    codes = torch.randint(0, 256, (2, NB, Hk, 16, D), generator=g, device="cuda", dtype=torch.uint8)
    for view in (torch.uint8, torch.float8_e4m3fn):
        a.zero_(), b.zero_()
        p.pa_gather_cache(a, b, codes[0].view(view), codes[1].view(view), slots, 0.013, 1.7)
        torch.cuda.synchronize()
        for got, pool, s in ((a, codes[0], 0.013), (b, codes[1], 1.7)):
            want = (pool.view(torch.float8_e4m3fn).float() * torch.tensor(s, device="cuda"))[at // 16, :, at % 16].to(dtype)
            assert same_nan(got[live], want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,Hk,T", [(64, 8, 20001), (128, 32, 3000), (64, 1, 70000)])
def test_many_rows_written_and_read_back(dtype, D, Hk, T):
    """More rows than the grids hold at once, a tenth of them padding: bit for bit."""
    p = pa()
    g = gen(T)
    NB = T // 16 + 20
    key, val = rand(g, (T, Hk, D), dtype, 3.0), rand(g, (T, Hk, D), dtype, 0.2)
    slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
    slots = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.1, torch.full_like(slots, -1), slots)
    kc, vc = (torch.full(p.int4_cache_shape(NB, Hk, D), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2))
    ek, ev = kc.clone(), vc.clone()
    p.pa_reshape_and_cache_int4(key, val, kc, vc, slots)
    a, b = torch.full_like(key, 5.0), torch.full_like(key, 5.0)
    p.pa_gather_cache(a, b, kc, vc, slots)
    torch.cuda.synchronize()
    live = slots >= 0
    for pool, want, x, back in ((kc, ek, key, a), (vc, ev, val, b)):
        codes, ends = ref.quantise(x)
        ref.put_rows(want, codes, ends, slots)
        assert torch.equal(pool, want)
        values = (codes.float() * ends[..., :1].float() + ends[..., 1:].float()).to(dtype)
        assert torch.equal(back[live], values[live]) and bool((back[~live] == 5.0).all())


def test_gather_flags_slots_past_the_pool():
    p = pa()
    pool = torch.zeros(p.int4_cache_shape(2, 4, 64), dtype=torch.uint8, device="cuda")
    a = torch.full((3, 4, 64), 9.0, dtype=torch.float16, device="cuda")
    b = a.clone()
    slots = torch.tensor([32, 1 << 45, 31], device="cuda")
    p.pa_gather_cache(a, b, pool, pool, slots)
    assert p.pa_device_error() == 4
    assert bool((a[:2] == 9.0).all()) and not a[2].any() and not b[2].any()
    p.pa_reshape_and_cache_int4(a, b, pool, pool.clone(), slots)
    assert p.pa_device_error() == 4


def test_int4_tokens_none_and_past_32_bits():
    """No tokens; and rows whose byte offset in the pool passes 2^32."""
    p = pa()
    Hk, D = 32, 128
    NB = (1 << 32) // (Hk * 1088) + 40
    kc, vc = (torch.zeros(p.int4_cache_shape(NB, Hk, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    none = torch.zeros((0, Hk, D), dtype=torch.float16, device="cuda")
    slots0 = torch.zeros(0, dtype=torch.int64, device="cuda")
    p.pa_reshape_and_cache_int4(none, none, kc, vc, slots0)
    p.pa_gather_cache(none, none, kc, vc, slots0)
    g = gen(4)
    T = 24
    key, val = rand(g, (T, Hk, D), torch.float16), rand(g, (T, Hk, D), torch.float16)
    slots = torch.cat((torch.arange(8), NB * 16 - 1 - torch.arange(16))).cuda()
    p.pa_reshape_and_cache_int4(key, val, kc, vc, slots)
    a, b = torch.empty_like(key), torch.empty_like(key)
    p.pa_gather_cache(a, b, kc, vc, slots)
    torch.cuda.synchronize()
    for got, x in ((a, key), (b, val)):
        c, e = ref.quantise(x)
        assert torch.equal(got, (c.float() * e[..., :1].float() + e[..., 1:].float()).half())
    # and attention over blocks at the pool's far end
    tables = torch.tensor([[NB - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([16], dtype=torch.int32, device="cuda")
    q = rand(g, (1, Hk, D), torch.float16)
    out = torch.empty_like(q)
    p.pa_decode_int4(out, q, kc, vc, tables, lens, 0.1, Hk, 16)
    torch.cuda.synchronize()
    want, slack = ref.attend(q[:, None], kc[-1:], vc[-1:], torch.zeros_like(tables), lens, 0.1)
    ref.near(out[:, None], want, slack, "far block")


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def batch(g, lens, Hk, group, D, dtype, q_len=1, spare=5, qk=2.0, **kw):
    """Pools, tables and queries; unused table entries are out of the pool, and
    blocks no sequence owns hold NaN scales."""
    S = len(lens)
    row = max(1, max(-(-n // 16) for n in lens) + 1)
    used = sum(-(-n // 16) for n in lens)
    NB = used + spare
    kc, vc = ref.random_pool(g, NB, Hk, D, **kw), ref.random_pool(g, NB, Hk, D, **kw)
    perm = torch.randperm(NB, generator=g, device="cuda")
    tables, at = torch.full((S, row), 1 << 30, dtype=torch.int32, device="cuda"), 0
    for i, n in enumerate(lens):
        b = -(-n // 16)
        tables[i, :b] = perm[at:at + b].int()
        if n % 16:  # rows behind the last token: NaN
            for pool in (kc, vc):
                ref.pool_views(pool)[1][perm[at + b - 1], :, n % 16:] = 0xFF
        at += b
    for pool in (kc, vc):
        ref.pool_views(pool)[1][perm[at:]] = 0xFF
    q = rand(g, (S, q_len, Hk * group, D), dtype, qk)
    return q, kc, vc, tables, torch.tensor(lens, dtype=torch.int32, device="cuda")


def run(q, kc, vc, tables, lens, scale, q_len=1, window=0, P=0, ks=1.0, vs=1.0, ext=False, order=None, maxlen=None):
    p = pa()
    n = int(lens.max()) if maxlen is None else maxlen
    out = torch.full_like(q, float("nan"))
    dims = p.ext_dims(q, kc, tables)
    if not ext and q_len == 1 and window == 0 and ks == vs == 1.0:
        bytes_ = p.pa_decode_workspace_size(dims, n, P)
        ws = torch.full((bytes_,), 0xFF, dtype=torch.uint8, device="cuda") if bytes_ else None
        p.pa_decode_int4(out[:, 0], q[:, 0], kc, vc, tables, lens, scale, kc.shape[1], n, P, ws)
    else:
        bytes_ = p.pa_decode_ext_workspace_size(dims, p.pa_decode_opts(q_len, window, ks, vs), n, P)
        ws = torch.full((bytes_,), 0xFF, dtype=torch.uint8, device="cuda") if bytes_ else None
        p.pa_decode_ext(out, q, kc, vc, tables, lens, scale, kc.shape[1], n, q_len, window, ks, vs, P, ws, seq_order=order)
    torch.cuda.synchronize()
    return out


def check(q, kc, vc, tables, lens, scale, what, **kw):
    out = run(q, kc, vc, tables, lens, scale, **kw)
    want, slack = ref.attend(q, kc, vc, tables, lens, scale, kw.get("q_len", 1), kw.get("window", 0), kw.get("ks", 1.0), kw.get("vs", 1.0))
    ref.near(out, want, slack, what)
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
def test_group_sizes_and_head_dims(dtype, D, group):
    g = gen(group + D)
    b = batch(g, [0, 1, 15, 16, 17, 31, 33, 250, 513, 1100], 2, group, D, dtype)
    for P in (0, 16, 48, 1104):
        check(*b, ref.scale_of(D), f"group {group} D {D} P {P}", P=P)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,q_len", [(1, 1), (1, 2), (1, 3), (1, 16), (2, 3), (4, 4), (8, 2), (4, 1), (16, 1), (5 - 4, 7)])
@pytest.mark.parametrize("window", [0, 1, 7, 16, 33, 300])
def test_query_tokens_and_windows(D, group, q_len, window):
    """Query rows that the window or the length leaves nothing for are zero."""
    g = gen(100 * group + 10 * q_len + window)
    b = batch(g, [0, 1, 2, 15, 16, 40, 129, 700], 2, group, D, torch.float16, q_len=q_len)
    for P in (0, 32):
        check(*b, ref.scale_of(D), f"P {P}", q_len=q_len, window=window, P=P, ext=True)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    rng = np.random.default_rng(900 + seed)
    g = gen(900 + seed)
    for _ in range(6):
        group = int(rng.choice([1, 2, 4, 8, 16]))
        q_len = int(rng.integers(1, 16 // group + 1))
        lens = [int(x) for x in rng.integers(0, int(rng.choice([20, 300, 3000])), size=int(rng.integers(1, 7)))]
        D, dtype = int(rng.choice([64, 128])), TYPES[int(rng.integers(2))]
        b = batch(g, lens, int(rng.choice([1, 3, 8])), group, D, dtype, q_len=q_len, level=float(rng.choice([0.01, 0.3, 2.0])))
        check(*b, ref.scale_of(D), f"{lens}", q_len=q_len, window=int(rng.choice([0, 0, 1, 50, 1000])), ext=True,
              P=int(rng.choice([0, 16, 64, 512])), ks=float(rng.choice([1.0, 0.5])), vs=float(rng.choice([1.0, 3.0])))


@pytest.mark.parametrize("S,Hk,most", [(4097, 1, 300), (5000, 2, 130), (300, 4, 100), (4096, 2, 200)])
def test_many_sequences(S, Hk, most):
    """Batches past the limit of the shared-out kernel, at it, and of short
    contexts; 60 sequences checked, the first and last among them."""
    g = gen(S)
    lens = [int(n) for n in torch.randint(0, most, (S,), generator=g, device="cuda")]
    lens[-1] = most
    q, kc, vc, tables, cl = batch(g, lens, Hk, 4, 64, torch.float16)
    out = run(q, kc, vc, tables, cl, 0.125)
    some = torch.cat((torch.randperm(S, generator=g, device="cuda")[:58], torch.tensor([0, S - 1], device="cuda")))
    want, slack = ref.attend(q[some], kc, vc, tables[some], cl[some], 0.125)
    ref.near(out[some], want, slack, f"{S} sequences")
    assert bool(out.isfinite().all())


def test_extreme_scales_and_queries():
    """V scales from 2^-100 to 2^100 in one sequence, rows of scale 0, K rows
    2^-60 small under queries 2^60 large, bf16."""
    g = gen(20)
    q, kc, vc, tables, lens = batch(g, [200, 37], 2, 4, 128, torch.bfloat16, qk=1.0)
    NB = kc.shape[0]
    vt, kt = ref.pool_views(vc)[1], ref.pool_views(kc)[1]
    s = torch.ldexp(torch.ones((NB, 2, 16), device="cuda"), torch.randint(-100, 101, (NB, 2, 16), generator=g, device="cuda")).to(torch.bfloat16)
    lo = (s.float() * -7).to(torch.bfloat16)
    zero = torch.rand((NB, 2, 16), generator=g, device="cuda") < 0.1
    s[zero] = 0.0
    vt.copy_(torch.stack((s, lo), -1).view(torch.uint8).view(NB, 2, 16, 4))
    check(q, kc, vc, tables, lens, 0.09, "V scales")
    e = kt.contiguous().view(torch.bfloat16).view(NB, 2, 16, 2)
    tiny = torch.where(e.isnan(), e, (e.float() * 2.0 ** -60).to(torch.bfloat16))
    kt.copy_(tiny.view(torch.uint8).view(NB, 2, 16, 4))
    check((q.float() * 2.0 ** 60).to(torch.bfloat16), kc, vc, tables, lens, 0.09, "large q", P=16)
    check((q.float() * 2.0 ** -60).to(torch.bfloat16), kc, vc, tables, lens, 0.09, "small q")
    check(torch.zeros_like(q), kc, vc, tables, lens, 0.09, "zero q")


def test_constant_rows_and_sharp_softmax():
    g = gen(21)
    q, kc, vc, tables, lens = batch(g, [300, 65], 1, 8, 64, torch.float16)
    for pool in (kc, vc):                                   # scale 0: a row of equal elements
        t = ref.pool_views(pool)[1]
        e = t.contiguous().view(torch.bfloat16).view(*t.shape[:3], 2)
        e[..., 0] = torch.where(e[..., 0].isnan(), e[..., 0], torch.zeros_like(e[..., 0]))
        t.copy_(e.view(torch.uint8).view(t.shape))
    check(q, kc, vc, tables, lens, 0.125, "constant rows")
    b = batch(g, [300, 65, 1000], 2, 4, 128, torch.float16, qk=12.0)   # logits of hundreds: one token takes all
    check(*b, 1.0, "sharp", P=32)
    check(*b, 1.0, "sharp")


def test_a_poisoned_row_reaches_only_its_readers():
    """A NaN row inside a context makes that KV head's outputs of that sequence NaN and nothing else."""
    g = gen(22)
    p = pa()
    q, kc, vc, tables, lens = batch(g, [40, 50], 2, 4, 64, torch.float16)
    clean = run(q, kc, vc, tables, lens, 0.125)
    x = torch.zeros((1, 2, 64), dtype=torch.float16, device="cuda")
    x[0, 1, 5] = float("nan")
    vt = ref.pool_views(vc)[1].clone()
    slot = (tables[0, 1].long() * 16 + 3).view(1)
    p.pa_reshape_and_cache_int4(torch.zeros_like(x), x, kc.clone(), vc, slot)
    out = run(q, kc, vc, tables, lens, 0.125)
    assert bool(out[0, 0, 4:].isnan().all())
    assert torch.equal(out[1], clean[1])
    ref.pool_views(vc)[1].copy_(vt)


@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("P", [0, 16])
def test_nan_queries_and_keys(group, P):
    """A NaN or infinite query element makes its own row NaN and no other; a
    NaN key row, even the only token of a sequence or of a partition, makes
    its KV head's rows of that sequence NaN."""
    g = gen(26)
    p = pa()
    b = batch(g, [1, 17, 200], 2, group, 128, torch.float16)
    q, kc, vc, tables, lens = b
    clean = run(*b, 0.09, P=P)
    bad = q.clone()
    bad[2, 0, 1, 7] = float("nan")
    bad[1, 0, group, 100] = float("inf")
    out = run(bad, kc, vc, tables, lens, 0.09, P=P)
    hit = torch.zeros(out.shape[:3], dtype=torch.bool, device="cuda")
    hit[2, 0, 1] = hit[1, 0, group] = True
    assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], clean[~hit])
    x = torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda")
    x[:, 1, 5] = float("nan")
    slots = torch.stack([tables[0, 0].long() * 16, tables[1, 1].long() * 16, tables[2, 5].long() * 16 + 9])
    p.pa_reshape_and_cache_int4(x, torch.zeros_like(x), kc, vc.clone(), slots)
    out = run(q, kc, vc, tables, lens, 0.09, P=P)
    assert bool(out[:, 0, group:].isnan().all())
    head0 = run(q, kc, vc, tables, lens, 0.09, P=P)[:, 0, :group]
    assert bool(head0.isfinite().all())


def test_bad_table_entries_and_lengths_are_flagged():
    g = gen(23)
    p = pa()
    q, kc, vc, tables, lens = batch(g, [64, 64, 64], 2, 2, 64, torch.float16)
    ok = run(q, kc, vc, tables, lens, 0.125)
    bad = tables.clone()
    bad[0, 1], bad[1, 2] = -3, kc.shape[0]
    out = run(q, kc, vc, bad, lens, 0.125)
    assert p.pa_device_error() == 1 and torch.equal(out[2], ok[2])
    short = torch.tensor([64, -5, 64], dtype=torch.int32, device="cuda")
    out = run(q, kc, vc, tables, short, 0.125)
    assert p.pa_device_error() == 2 and not out[1].any() and torch.equal(out[0], ok[0])
    long = torch.tensor([64, 64, 1 << 30], dtype=torch.int32, device="cuda")
    out = run(q, kc, vc, tables, long, 0.125, maxlen=64)
    assert p.pa_device_error() & 2 and torch.equal(out[:2], ok[:2])


def test_seq_order_and_repeatability():
    g = gen(24)
    lens = [int(n) for n in torch.randint(1, 2000, (24,), generator=g, device="cuda")]
    b = batch(g, lens, 2, 4, 128, torch.bfloat16)
    a = run(*b, 0.09, ext=True)
    order = torch.randperm(24, generator=g, device="cuda").int()
    assert torch.equal(run(*b, 0.09, ext=True, order=order), a)
    assert torch.equal(run(*b, 0.09), a)
    for P in (16, 256):
        assert torch.equal(run(*b, 0.09, P=P), run(*b, 0.09, P=P))


def test_noncontiguous_and_wrong_types_refused():
    g = gen(25)
    p = pa()
    q, kc, vc, tables, lens = batch(g, [20, 20], 2, 2, 64, torch.float16)
    out = torch.empty_like(q[:, 0])
    with pytest.raises(ValueError):
        p.pa_decode_int4(out, q[:, 0], kc[:, :1], vc[:, :1], tables, lens, 0.1, 1, 20)
    with pytest.raises(TypeError):
        p.pa_decode_int4(out, q[:, 0], kc, vc, tables.long(), lens, 0.1, 2, 20)
    with pytest.raises(TypeError):
        p.pa_decode_int4(out, q[:, 0], kc.view(-1, 2, 18, 32), vc, tables, lens, 0.1, 2, 20)
    x = torch.zeros((4, 2, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        p.pa_reshape_and_cache_int4(x, x, kc, vc, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        p.pa_reshape_and_cache_int4(x, x, kc, vc, torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        p.pa_gather_cache(x[:, :1].contiguous(), x, kc, vc, torch.zeros(4, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------------------
# blocks, steps, graphs
# ---------------------------------------------------------------------------
def test_copy_and_swap_blocks():
    g = gen(30)
    p = pa()
    for Hk, D in ((3, 64), (8, 128)):
        kc, vc = ref.random_pool(g, 20, Hk, D), ref.random_pool(g, 20, Hk, D)
        ek, ev = kc.clone(), vc.clone()
        pairs = torch.tensor([[0, 10], [3, 11], [7, 19]], device="cuda")
        p.pa_copy_blocks([kc], [vc], pairs)
        for e in (ek, ev):
            e[pairs[:, 1]] = e[pairs[:, 0]]
        assert torch.equal(kc, ek) and torch.equal(vc, ev)
        hk, hv = (torch.zeros((6, Hk, 8 * D + 64), dtype=torch.uint8).pin_memory() for _ in range(2))
        p.pa_swap_blocks(kc, vc, hk, hv, torch.tensor([[19, 2], [4, 0]], device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(hk[2], ek[19].cpu()) and torch.equal(hv[0], ev[4].cpu()) and not hk[1].any()
        p.pa_swap_blocks(hk, hv, kc, vc, torch.tensor([[2, 5]], device="cuda"))
        ek[5], ev[5] = ek[19], ev[19]
        assert torch.equal(kc, ek) and torch.equal(vc, ev)


@pytest.mark.parametrize("kind", ["int4", "16", "fp8"])
def test_decode_steps_with_rotation(kind):
    """Prompts and decode steps as a server runs them: rotate, append, attend;
    the cache's own rows, read back, are what 64-bit attention uses."""
    p = pa()
    g = gen(31)
    S, H, Hk, D, NB, dtype = 3, 8, 2, 128, 40, torch.bfloat16
    f, m = p.pa_rope_frequencies(D, 10000.0, "yarn", factor=4.0, original_context=256)
    f = f.cuda()
    if kind == "int4":
        kc, vc = (torch.full(p.int4_cache_shape(NB, Hk, D), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    elif kind == "fp8":
        kc, vc = (torch.full((NB, Hk, 16, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        kc, vc = (torch.full((NB, Hk, 16, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = (0.02, 0.02) if kind == "fp8" else (1.0, 1.0)
    tables = torch.randperm(NB, generator=g, device="cuda")[:S * 12].view(S, 12).int()
    lens = [33, 1, 100]

    def append(rows):
        """rows: (sequence, position) of each new token; returns its queries."""
        T = len(rows)
        qkv = rand(g, (T, H + 2 * Hk, D), dtype)
        pos = torch.tensor([r[1] for r in rows], device="cuda")
        slots = torch.stack([tables[s, n // 16].long() * 16 + n % 16 for s, n in rows])
        q = torch.empty((T, H, D), dtype=dtype, device="cuda")
        p.pa_rope_and_cache(q, qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], kc, vc, slots, pos, f, magnitude=m, k_scale=ks, v_scale=vs)
        ref.near(q, ref.rotate(qkv[:, :H], pos, f, False, m), ref.rotate_bound(qkv[:, :H], f, False, m), "q")
        return q

    append([(s, n) for s in range(S) for n in range(lens[s])])
    for _ in range(3):
        q = append([(s, lens[s]) for s in range(S)])
        lens = [n + 1 for n in lens]
        cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        args = (out, q, kc, vc, tables, cl)
        scale = ref.scale_of(D)
        if kind == "int4":
            p.pa_decode_int4(*args, scale, Hk, max(lens))
        elif kind == "fp8":
            p.pa_decode_fp8(*args, scale, ks, vs, Hk, max(lens))
        else:
            p.pa_decode(*args, scale, Hk, max(lens))
        for s in range(S):
            at = torch.arange(lens[s], device="cuda")
            slots = tables[s].long()[at // 16] * 16 + at % 16
            K, V = (torch.empty((lens[s], Hk, D), dtype=dtype, device="cuda") for _ in range(2))
            p.pa_gather_cache(K, V, kc, vc, slots, ks, vs)
            x = torch.einsum("hgd,thd->hgt", q[s].double().view(Hk, H // Hk, D), K.double()) * scale
            want = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), V.double()).reshape(H, D)
            # the read-back rounds K and V to bf16 (2^-8): logits move by at most 2^-8 c sum|q k|, outputs by twice
            # that times max|V|, and by 2^-8 max|V|; the 16-bit and FP8 kernels round weights to bf16 or finer (2^-8)
            d = 2.0 ** -8 * scale * float(torch.einsum("hgd,thd->hgt", q[s].double().abs().view(Hk, H // Hk, D), K.double().abs()).max())
            tol = (2 * d + 3 * 2.0 ** -8) * float(V.abs().max())
            assert float((out[s].double() - want).abs().max()) <= tol


def test_graphs_with_a_shared_workspace_and_streams():
    """Two captured steps that share a workspace, replayed in turn, give what
    eager calls give; two streams with workspaces of their own run at once."""
    p = pa()
    g = gen(32)
    a = batch(g, [1500, 700, 20], 2, 8, 128, torch.float16)
    b = batch(g, [900, 1900], 4, 2, 64, torch.float16)
    size = max(p.pa_decode_workspace_size(p.ext_dims(x[0], x[1], x[3]), 2000 if x[3].shape[1] * 16 >= 2000 else x[3].shape[1] * 16, 64) for x in (a, b))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(x[0][:, 0]) for x in (a, b)]

    def call(x, out, ws, stream=None):
        q, kc, vc, tables, lens = x
        p.pa_decode_int4(out, q[:, 0], kc, vc, tables, lens, 0.1, kc.shape[1], 1900 if tables.shape[1] * 16 >= 1900 else tables.shape[1] * 16, 64, ws, stream=stream)

    want = []
    for x, o in zip((a, b), outs):
        call(x, o, ws)
        torch.cuda.synchronize()
        want.append(o.clone())
    graphs = []
    for x, o in zip((a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(x, o, ws)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(ws) for _ in range(2)]
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for x, o, st, w in zip((a, b), outs, streams, spaces):
            call(x, o, w, st)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_inputs_written_by_the_kernel_in_front():
    """A captured loop whose torch kernels change positions, slots, lengths and
    queries right in front of the calls, two batches sharing a workspace with
    automatic shares: every step as a synchronised eager one gives it."""
    p = pa()
    g = gen(33)
    steps, H, Hk, D = 24, 8, 2, 128
    f, _ = p.pa_rope_frequencies(D)
    f = f.cuda()
    lens0 = [[2000, 130, 1], [900, 700, 33, 5, 256]]
    sets = []
    for lens in lens0:
        S = len(lens)
        rows = 2064 // 16
        NB = S * rows
        kc, vc = ref.random_pool(g, NB, Hk, D), ref.random_pool(g, NB, Hk, D)
        tables = torch.randperm(NB, generator=g, device="cuda").int().view(S, rows)
        news = [rand(g, (steps, S, h, D), torch.bfloat16) for h in (H, Hk, Hk)]
        sets.append(dict(kc=kc, vc=vc, tables=tables, news=news, S=S, first=torch.tensor(lens, dtype=torch.int32, device="cuda")))
    size = max(p.pa_decode_workspace_size(p.dims_of(x["news"][0][0], x["kc"], x["tables"]), 2064) for x in sets)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def loop(sync):
        outs = []
        state = []
        for x in sets:
            state.append(dict(kc=x["kc"].clone(), vc=x["vc"].clone(), lens=x["first"].clone(), pos=torch.zeros(x["S"], dtype=torch.int64, device="cuda"),
                              slots=torch.zeros(x["S"], dtype=torch.int64, device="cuda"), q=torch.empty_like(x["news"][0][0]),
                              rq=torch.empty_like(x["news"][0][0]), k=torch.empty_like(x["news"][1][0]), v=torch.empty_like(x["news"][1][0])))

        def body():
            for t in range(steps):
                for x, s in zip(sets, state):
                    for name, new in zip("qkv", x["news"]):
                        s[name].copy_(new[t])
                    at = s["lens"].long()
                    s["slots"].copy_(x["tables"].gather(1, (at // 16)[:, None])[:, 0].long() * 16 + at % 16)
                    s["pos"].copy_(at)
                    p.pa_rope_and_cache(s["rq"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"], f)
                    s["lens"].add_(1)
                    out = torch.empty_like(s["q"])
                    if sync:
                        torch.cuda.synchronize()
                    p.pa_decode_int4(out, s["rq"], s["kc"], s["vc"], x["tables"], s["lens"], D ** -0.5, Hk, 2064, 0, ws)
                    if sync:
                        torch.cuda.synchronize()
                    outs.append(out)
        return body, outs, state

    body, want, _ = loop(True)
    body()
    body, got, _state = loop(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    graph.replay()
    torch.cuda.synchronize()
    assert len(got) == len(want) == 2 * steps
    for a, b in zip(got, want):
        assert torch.equal(a, b)
