"""The query's integers in 4-bit decode: what the header states of them against
arithmetic on the CPU, and the kernels against what it states."""
import os
import re

import pytest
import torch

import kv4_ref as ref
import kv4_weights_ref as kw

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pa.h")


def stated():
    """(1 / error relative to the largest, reach of exact fp16 elements, of bf16 ones) as the header has them."""
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER).read())
    m = re.search(r"every element to within 1 / (\d+) of the row's largest \|q\| \(exact for fp16 elements down to a (\d+)th of it, for bf16 ones down to a (\d+)th\)", text)
    assert m, "the header does not state the query's accuracy in these words"
    return tuple(int(x) for x in m.groups())


def integers(x, largest):
    """x in units of a row whose largest element is `largest` (float64 tensors): the largest becomes 16320 .. 32639."""
    _, e = torch.frexp(largest)
    top = torch.ldexp(largest, 15 - e)
    e = e + (top > 32639.0)
    return torch.ldexp(x, 15 - e)


@pytest.mark.parametrize("dtype,which", [(torch.float16, 1), (torch.bfloat16, 2)])
def test_the_stated_reach_is_exact(dtype, which):
    bits = {torch.float16: 10, torch.bfloat16: 7}[dtype]
    mantissas = 1.0 + torch.arange(2 ** bits, dtype=torch.float64) / 2 ** bits
    error, reach = stated()[0], stated()[which]
    beyond = False
    for largest in mantissas:
        for down in range(0, 9):
            x = mantissas * 2.0 ** -down
            x = x[x <= largest]
            y = integers(x, largest)
            v = torch.round(y)
            hi = torch.floor((v + 128) / 256)
            lo = v - 256 * hi
            assert bool(((hi >= -128) & (hi <= 127) & (lo >= -128) & (lo <= 127)).all())
            hi = torch.floor((-v + 128) / 256)
            assert bool(((hi >= -128) & (hi <= 127)).all())
            off = (v - y).abs() / integers(largest[None], largest)
            assert bool((off <= 1.0 / error).all())
            inside = x * reach >= largest
            assert bool((v == y)[inside].all())
            beyond |= bool((v != y)[(x * 2 * reach >= largest) & ~inside].any())
    assert beyond  # twice as far is not


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 2, 8, 16])
@pytest.mark.parametrize("dtype,which,factor", [(torch.float16, 1, 128.0), (torch.bfloat16, 2, 512.0)])
def test_elements_within_reach_are_exact_on_the_gpu(dtype, which, factor, group):
    """Token t has one code, 15 at dim t: its logit is factor q_t.  The q_t lie at the end of the stated reach
    under an element of 1; a logit is then off by fp32 roundings alone: d = 2 (D + 8) 2^-24 |x| + 2^-22 (3 max|x| +
    6), the output by (e^(2 d) - 1) A + (2^-19 + 15 2^-22 + 7.5 2^-11 (more than 4 rows) + 3 f) A, A = 15 the largest
    |V|, f = 1.1 (n + 32) 2^-24."""
    from gpu_util import require_gpu
    require_gpu()
    from paged_kv_cache_424_b200 import binding as p
    reach, D = stated()[which], 128
    n = D - 1
    g = torch.Generator("cuda")
    g.manual_seed(group)
    kc, vc = kw.pools(g, n, 1, D)
    rows = ref.pool_views(kc)[0]
    rows.zero_()
    for t in range(n):
        rows[t // 16, 0, t % 16, t // 2] = 15 << (4 * (t % 2))
    N = kc.shape[0] * 16
    kw.set_rows(kc, torch.ones(N), torch.zeros(N))
    power = 2.0 ** -reach.bit_length()  # below the reach; what is beyond it is left out
    bits = {torch.float16: 10, torch.bfloat16: 7}[dtype]
    step = torch.randint(0, 2 ** bits, (group, D), generator=g, device="cuda")
    q = power * (1.0 + step.double() / 2 ** bits)
    q = torch.where(q * reach >= 1.0, q, torch.full_like(q, 2 * power)).to(dtype)
    q[:, D - 1] = 1.0
    scale = factor / 15.0
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty((1, group, D), dtype=dtype, device="cuda")
    p.pa_decode_int4(out, q[None], kc, vc, table, lens, scale, 1, n)
    torch.cuda.synchronize()
    x = 15.0 * q.double()[:, :n] * torch.tensor(scale, dtype=torch.float32).double().item()
    V = ref.values(vc)[:, 0].reshape(-1, D)[:n]
    want = torch.softmax(x, -1) @ V
    top = float(x.abs().max())
    d = 2 * (D + 8) * 2.0 ** -24 * top + 2.0 ** -22 * (3 * top + 6)
    slack = (float(torch.expm1(torch.tensor(2 * d, dtype=torch.float64))) + 2.0 ** -19 + 15 * 2.0 ** -22 +
             (7.5 * 2.0 ** -11 if group > 4 else 0.0) + 3 * 1.1 * (n + 32) * 2.0 ** -24) * 15.0
    ref.near(out[0], want, torch.full_like(want, slack), "logits of single elements")
    assert p.pa_device_error() == 0
