"""Plain 64-bit forms of the rotary, 4-bit cache and read-back operators, and
the error bounds the GPU tests hold the kernels to.

A rounding to a type is off by at most half a step: eps / 2 relative (bf16
2^-8, fp16 2^-11, fp32 2^-24, E4M3 2^-4).
"""
import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}
# half the distance between the smallest numbers of a type (its rounding error near zero)
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float8_e4m3fn: 2.0 ** -10}


def rotate(x, positions, inv_freq, interleaved, magnitude=1.0, inverse=False):
    """float64 rotation of [tokens, heads, D] rows."""
    x = x.double()
    h = inv_freq.numel()
    th = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(th) * magnitude, torch.sin(th) * magnitude * (-1.0 if inverse else 1.0)
    out = x.clone()
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def rotate_bound(x, inv_freq, interleaved, magnitude=1.0):
    """Error of the rotation in fp32 before the final rounding: cos and sin are
    each off by half a step of fp32 (the angle in fp64 adds far less), so are
    the two products and their sum: at most 3 half steps of m (|a| + |b|)."""
    x = x.double().abs()
    h = inv_freq.numel()
    out = torch.zeros_like(x)
    ia, ib = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    both = (x[..., ia] + x[..., ib]) * abs(magnitude) * 3.0 * 2.0 ** -24 + 2.0 ** -148
    out[..., ia] = both
    out[..., ib] = both
    return out


def near(got, want, slack, what):
    """got (16-bit) is want rounded once, want itself known to within slack."""
    g = got.double()
    bound = slack + HALF_STEP[got.dtype] * (want.abs() + slack) + TINY[got.dtype]
    bad = ~((g - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} values off, worst {float((g - want).abs().max()):.3e}"


def quantise(x):
    """fp32 rows [.., D] -> (codes uint8 [.., D], ends bf16 [.., 2]): the written rule, operation by operation."""
    x = x.float()
    low = x.amin(-1).to(torch.bfloat16)
    lowf = low.float()
    fifteen = torch.full((), 15.0, device=x.device)
    scale = ((x.amax(-1) - lowf) / fifteen).to(torch.bfloat16)
    bad = ~torch.isfinite(x).all(-1) | ~torch.isfinite(scale.float())
    y = torch.round((x - lowf[..., None]) / scale.float()[..., None]).clamp(0.0, 15.0)
    codes = torch.where((scale.float()[..., None] != 0) & ~bad[..., None], y, torch.zeros_like(y)).to(torch.uint8)
    nan = torch.full_like(low, float("nan"))
    return codes, torch.stack((torch.where(bad, nan, scale), torch.where(bad, nan, low)), -1)


def pool_views(pool):
    """(codes [NB, Hk, 16, D / 2], ends uint8 [NB, Hk, 16, 4]) views of a 4-bit pool."""
    D = (pool.shape[2] - 64) // 8
    return pool[:, :, :8 * D].unflatten(2, (16, D // 2)), pool[:, :, 8 * D:].unflatten(2, (16, 4))


def put_rows(pool, codes, ends, slots):
    """Writes quantised rows [T, Hk, ..] where slots (a CPU or CUDA int64 tensor) are inside the pool."""
    rows, tail = pool_views(pool)
    live = (slots >= 0) & (slots < pool.shape[0] * 16)
    at = slots[live]
    rows[at // 16, :, at % 16] = codes[live][..., 0::2] | (codes[live][..., 1::2] << 4)
    tail[at // 16, :, at % 16] = ends[live].contiguous().view(torch.uint8).unflatten(-1, (-1, 4)).squeeze(-2)


def values(pool, dtype=torch.float64):
    """Every element of a pool: [NB, Hk, 16, D]."""
    codes, tail = pool_views(pool)
    e = tail.contiguous().view(torch.bfloat16).to(dtype)
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(dtype)
    return u * e[..., :1] + e[..., 1:]


def random_pool(gen, NB, Hk, D, spread=0.3, level=0.3):
    """A pool of random codes; scales and lowest values as rows of normal numbers have them."""
    pool = torch.randint(0, 256, (NB, Hk, 8 * D + 64), generator=gen, device="cuda", dtype=torch.uint8)
    s = (level * torch.exp(spread * torch.randn((NB, Hk, 16), generator=gen, device="cuda"))).to(torch.bfloat16)
    lo = (s.float() * (-7.5 + torch.randn((NB, Hk, 16), generator=gen, device="cuda"))).to(torch.bfloat16)
    pool_views(pool)[1].copy_(torch.stack((s, lo), -1).view(torch.uint8).view(NB, Hk, 16, 4))
    return pool


def query_integers(q):
    """Rows [.., D] as the kernel takes them: integers (largest in 2^13 .. 2^14 - 1) under a power of two per row."""
    q = q.double()
    _, e = torch.frexp(q.abs().amax(-1, keepdim=True))
    up = torch.ldexp(torch.ones_like(q[..., :1]), (14 - e).clamp(max=120))
    return torch.round(q * up).clamp(max=16383.0) / up


def attend(q, k_pool, v_pool, tables, lens, scale, q_len=1, window=0, k_scale=1.0, v_scale=1.0):
    """float64 attention [S, q_len, H, D] and, per output, the bound of the
    kernel's error before the output's own rounding.

    With p the weights (sum 1), s_t, l_t a V row's scale and low and r = q . u:
      - the weight times the V scale is rounded to fp16 (half a step, 2^-11;
        numbers below its normal range lie under 2^-24 of the largest weight
        times scale); what a rounding takes from a weight is given back at
        the middle code, so a code u carries at most |u - 7.5| <= 7.5 of it:
        (2^-11 + 2^-20) 7.5 max|s_t|;
      - a logit c (s (q . u) + l sum(q)) is a sum of D products in fp32 in any
        order, whose terms are at most c |s| 15 sum|q|, and l sum(q) likewise:
        with 2 (D + 8) half steps of fp32 for sums, products, the query's own
        scaling and the exponential, d = 2 (D + 8) 2^-24 c (15 max|s| +
        max|l|) sum|q| plus 2^-21 of the largest |logit| and as much again
        for the exponential.  The query enters as integers under a power of
        two (`query_integers`): with e_i what that takes from element i, a
        logit moves by |sum_i e_i (s u_i + l)| <= (15 max|s| + max|l|)
        c sum|e|.  Moving each logit by at most d moves the output by at most
        (e^(2 d) - 1) max|v|.
      - sums of weights and outputs over n tokens in fp32: (n / 16 + 64) half
        steps at the most of the sum of magnitudes, max(15 |s| + |l|).
    """
    S, QL, H, D = q.shape
    Hk = k_pool.shape[1]
    g = H // Hk
    kv, vv = values(k_pool) * k_scale, values(v_pool) * v_scale
    ke, ve = (pool_views(x)[1].contiguous().view(torch.bfloat16).double() for x in (k_pool, v_pool))
    out = torch.zeros((S, QL, H, D), dtype=torch.float64, device=q.device)
    slack = torch.zeros_like(out)
    for i in range(S):
        n = int(lens[i])
        blocks = tables[i, :-(-n // 16)].long()
        for j in range(QL):
            p = n - QL + j
            lo = max(0, p - window + 1) if window > 0 else 0
            if p < lo:
                continue
            at = torch.arange(lo, p + 1, device=q.device)
            b, o = blocks[at // 16], at % 16
            K, V = kv[b, :, o], vv[b, :, o]                      # [n, Hk, D]
            qq = q[i, j].double().reshape(Hk, g, D)
            x = torch.einsum("hgd,thd->hgt", qq, K) * scale
            w = torch.softmax(x, -1)
            out[i, j] = torch.einsum("hgt,thd->hgd", w, V).reshape(H, D)
            sk, lk = ke[b, :, o, 0].abs().amax(0) * k_scale, ke[b, :, o, 1].abs().amax(0) * k_scale
            sv, lv = ve[b, :, o, 0].abs().amax(0) * v_scale, ve[b, :, o, 1].abs().amax(0) * v_scale
            qs = qq.abs().sum(-1) * abs(scale)                   # [Hk, g]
            lost = (qq - query_integers(qq)).abs().sum(-1) * abs(scale)
            d = (15 * sk + lk)[:, None] * (2 * (D + 8) * 2.0 ** -24 * qs + lost) + 2.0 ** -20 * x.abs().amax(-1)
            top = (15 * sv + lv)[:, None]
            e = (2.0 ** -11 + 2.0 ** -20) * 7.5 * sv[:, None] + torch.expm1(2 * d) * top + \
                (len(at) / 16 + 64) * 2.0 ** -24 * top
            slack[i, j] = e.reshape(H, 1).expand(H, D)
    return out, slack


def scale_of(D):
    return 1.0 / math.sqrt(D)
