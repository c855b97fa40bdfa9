"""4-bit decode where the rounding of softmax weights would show: many small
weights beside a large one, V scales far above the others' at tokens of no
weight or that a row does not see, the second part of a split weight.  Bounds in
which each token counts by its weight (kv4_weights_ref.attend)."""
import math

import pytest
import torch

import kv4_ref as ref
import kv4_weights_ref as kw
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
LOG2E = math.log2(math.e)


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    from paged_kv_cache_424_b200 import build
    build.build()
    from paged_kv_cache_424_b200 import binding
    assert binding.pa_device_error() == 0, "device error word set before the test"
    yield
    assert binding.pa_device_error() == 0, "a kernel flagged a device error"


def gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def run(q, kc, vc, tables, lens, scale, q_len=1, window=0, P=0):
    from paged_kv_cache_424_b200 import binding as p
    n = int(lens.max())
    out = torch.full_like(q, float("nan"))
    bytes_ = p.pa_decode_ext_workspace_size(p.ext_dims(q, kc, tables), p.pa_decode_opts(q_len, window, 1.0, 1.0), n, P)
    ws = torch.full((max(bytes_, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    p.pa_decode_ext(out, q, kc, vc, tables, lens, scale, kc.shape[1], n, q_len, window, 1.0, 1.0, P, ws)
    torch.cuda.synchronize()
    return out


def check(q, kc, vc, n, scale, what, q_len=1, window=0, P=0, seqs=1):
    """One sequence over the pools' blocks in order, or `seqs` that share them (so that a warp has a context whole)."""
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")
    tables = table[None].expand(seqs, -1).contiguous()
    lens = torch.full((seqs,), n, dtype=torch.int32, device="cuda")
    out = run(q[None].expand(seqs, -1, -1, -1).contiguous(), kc, vc, tables, lens, scale, q_len, window, P)
    want, slack = kw.attend(q, kc, vc, table, n, scale, q_len, window)
    for i in {0, seqs // 2, seqs - 1}:
        ref.near(out[i], want, slack, f"{what}, sequence {i}")


def queries(q_len, group, D, dtype=torch.float16, Hk=1):
    """Rows whose elements add up to 1 exactly."""
    return torch.full((q_len, Hk * group, D), 1.0 / D, dtype=dtype, device="cuda")


ROWS = [(1, 1), (4, 1), (1, 3), (8, 1), (2, 3), (16, 1), (4, 4)]  # group, query tokens: 1, 2 and 4 tiles of rows


@pytest.mark.parametrize("group,q_len", ROWS)
@pytest.mark.parametrize("n,seqs,bits", [(4096, 3000, 24.6), (32768, 3000, 24.6), (32768, 3000, 29.0), (4096, 1, 24.6)])
def test_many_small_weights_beside_a_large_one(group, q_len, n, seqs, bits):
    """Token 5 holds the maximum and its row is all 0, all others have 2^-bits of it; all their codes 15, then all 1."""
    D = 64
    for byte in (0xFF, 0x11):
        kc, vc = kw.pools(gen(1), n, 1, D)
        ref.pool_views(vc)[0].fill_(byte)
        ref.pool_views(vc)[0][0, :, 5] = 0
        low = torch.full((kc.shape[0] * 16,), -1.0)
        low[5] = 0.0
        kw.set_rows(kc, torch.zeros_like(low), low)
        kw.set_rows(vc, torch.full_like(low, 0.75), torch.zeros_like(low))
        check(queries(q_len, group, D), kc, vc, n, bits / LOG2E, f"codes {byte:#x}", q_len=q_len, seqs=seqs)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group,q_len", ROWS)
@pytest.mark.parametrize("where", ["first", "middle", "last", "before the maximum"])
def test_large_scale_without_weight(dtype, group, q_len, where):
    """A V row 2^14 to 2^100 times the others' that its logit keeps out (2^-29 of the others by weight times scale); the others' logits about equal."""
    n, D = 1500, 64
    for ratio in (14, 17, 20, 60, 100):
        g = gen(ratio)
        kc, vc = kw.pools(g, n, 1, D)
        N = kc.shape[0] * 16
        low = torch.rand((N,), generator=g, device="cuda").cpu()
        if where == "before the maximum":  # tokens of growing weight behind it
            low = torch.linspace(-40.0, 0.0, N)
        at = {"first": 0, "middle": 700, "last": n - q_len, "before the maximum": 3}[where]
        low[at] = -20.0 - 0.7 * ratio
        kw.set_rows(kc, torch.zeros(N), low)
        s = 1.0 + torch.rand((N,), generator=g, device="cuda").cpu()
        s[at] = 2.0 ** ratio
        kw.set_rows(vc, s, -7.5 * s)
        for P in (0, 256):
            check(queries(q_len, group, D, dtype), kc, vc, n, 1.0, f"2^{ratio} {where} P {P}", q_len=q_len, P=P)


@pytest.mark.parametrize("group,q_len", [(1, 2), (1, 4), (2, 2), (2, 4), (4, 4), (1, 16)])
def test_large_scale_that_only_a_later_query_sees(group, q_len):
    """The last token's V row is 2^17 (2^100) times the others': only the last query token attends to it; and one
    that a window leaves to the first query token alone."""
    D, n = 128, 333
    for ratio in (17, 100):
        for at, window in ((n - 1, 0), (n - q_len - 19, 20)):
            g = gen(ratio)
            kc, vc = kw.pools(g, n, 2, D)
            N = kc.shape[0] * 16
            kw.set_rows(kc, torch.zeros(N), torch.rand((N,), generator=g, device="cuda").cpu())
            s = 1.0 + torch.rand((N,), generator=g, device="cuda").cpu()
            s[at] = 2.0 ** ratio
            kw.set_rows(vc, s, -7.5 * s)
            q = queries(q_len, group, D, torch.bfloat16, 2)
            for P in (0, 64):
                check(q, kc, vc, n, 1.0, f"2^{ratio} at {at} P {P}", q_len=q_len, window=window, P=P)


@pytest.mark.parametrize("group,q_len", ROWS)
@pytest.mark.parametrize("spread", [8.0, 40.0])
def test_scales_and_logits_over_wide_ranges(group, q_len, spread):
    """V scales over 2^+-spread against logits over about as many powers of two, unrelated; bf16."""
    D = 64
    for seed, n in ((1, 77), (2, 1000), (3, 4000)):
        g = gen(seed)
        kc, vc = kw.pools(g, n, 1, D)
        N = kc.shape[0] * 16
        kw.set_rows(kc, torch.zeros(N), torch.randn((N,), generator=g, device="cuda").cpu())
        s = torch.exp2(spread * (2 * torch.rand((N,), generator=g, device="cuda").cpu() - 1))
        kw.set_rows(vc, s, -7.5 * s)
        for scale in (0.3, spread / 2):
            check(queries(q_len, group, D, torch.bfloat16), kc, vc, n, scale, f"n {n} scale {scale}", q_len=q_len)


@pytest.mark.parametrize("group,q_len", ROWS)
@pytest.mark.parametrize("level", [110, 60, 0, -60, -85])
def test_levels_and_constant_rows(group, q_len, level):
    """All V rows near 2^level; the same with every third row constant (scale 0), some of those 2^16 larger; bf16."""
    D = 64
    for seed, n in ((4, 50), (5, 900)):
        for constant in (False, True):
            g = gen(seed)
            kc, vc = kw.pools(g, n, 1, D)
            N = kc.shape[0] * 16
            kw.set_rows(kc, torch.zeros(N), torch.randn((N,), generator=g, device="cuda").cpu())
            s = 2.0 ** level * (1.0 + torch.rand((N,), generator=g, device="cuda").cpu())
            low = -7.5 * s
            if constant:
                s[::3] = 0.0
                if level < 110:
                    low[::9] *= 2.0 ** 16
            kw.set_rows(vc, s, low)
            for P in (0, 64):
                check(queries(q_len, group, D, torch.bfloat16), kc, vc, n, 2.0, f"n {n} constant {constant} P {P}", q_len=q_len, P=P)


@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("D", [64, 128])
def test_second_part_of_a_weight(group, D):
    """Near-equal weights whose products with the scales need more than 11 bits, V around 0: what fp16 weights alone
    would leave is several times the bound."""
    n, g = 40, gen(D)
    kc, vc = kw.pools(g, n, 2, D)
    N = kc.shape[0] * 16
    kw.set_rows(kc, torch.zeros(N), torch.rand((N,), generator=g, device="cuda").cpu())
    s = 1.0 + torch.rand((N,), generator=g, device="cuda").cpu()
    kw.set_rows(vc, s, -7.5 * s)
    q = queries(1, group, D, torch.float16, 2)
    check(q, kc, vc, n, 0.25, "split weights")
    # the same weights rounded to fp16 are outside the bound (arithmetic of the oracle alone)
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")
    want, slack = kw.attend(q, kc, vc, table, n, 0.25)
    K, V = (ref.values(x).permute(0, 2, 1, 3).reshape(-1, 2, D)[:n] for x in (kc, vc))
    ends = ref.pool_views(vc)[1].contiguous().view(torch.bfloat16).double().permute(0, 2, 1, 3).reshape(-1, 2, 2)[:n]
    x = torch.einsum("hgd,thd->hgt", q[0].double().view(2, group, D), K) * 0.25
    pr = torch.exp(x - x.amax(-1, keepdim=True))
    w = (pr * ends[:, :, 0].t()[:, None]).half().double()
    codes = (V - ends[..., 1:]) / ends[..., :1]
    out = (torch.einsum("hgt,thd->hgd", w, codes) + torch.einsum("hgt,th->hg", pr, ends[..., 1])[..., None]) / pr.sum(-1, keepdim=True)
    far = (out.reshape(1, 2 * group, D) - want).abs() - slack - 2.0 ** -11 * (want.abs() + slack) - 2.0 ** -25
    assert bool((far > 0).any())


@pytest.mark.parametrize("group,q_len", ROWS)
@pytest.mark.parametrize("P", [0, 4096])
def test_rows_of_zeros(group, q_len, P):
    """V rows of nothing but zeros under rising logits give zeros; a last row that is not zero gives its share, whether
    it holds the softmax or a 2^-20 of it."""
    D, n = 64, 30000
    g = gen(P)
    kc, vc = kw.pools(g, n, 1, D)
    N = kc.shape[0] * 16
    low = torch.linspace(-30.0, 30.0, N)
    zeros = torch.zeros(N)
    kw.set_rows(kc, zeros, low)
    kw.set_rows(vc, zeros, zeros)
    q = queries(q_len, group, D, torch.bfloat16)
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    out = run(q[None], kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 1.0, q_len, 0, P)
    assert not out.any()
    for at, logit in ((n - q_len, 45.0), (n - q_len, 16.0), (0, 45.0), (0, 16.0)):
        k2, s = low.clone(), zeros.clone()
        k2[at], s[at] = logit, 1.0
        kw.set_rows(kc, zeros, k2)
        kw.set_rows(vc, s, -7.5 * s)
        check(q, kc, vc, n, 1.0, f"one row at {at}, logit {logit}", q_len=q_len, P=P)
