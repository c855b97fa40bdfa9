"""Attention over a 4-bit cache in 64 bits with a bound of the kernel's error
in which every token counts by its softmax weight, and pools that put the
weights where a rounding of theirs would show."""
import torch

import kv4_ref as ref


def attend(q, k_pool, v_pool, table, n, scale, q_len=1, window=0):
    """float64 attention [q_len, H, D] of one sequence of n tokens, and the
    bound of the kernel's error per output before the output's own rounding.
    With softmax weights w_t (sum 1), s_t and lo_t a V row's scale and low, u_t
    its code, S = sum w_t |s_t|, T = max w_t |s_t|, A = sum_t w_t (|s_t| u_t + |lo_t|):
      - weights w_t s_t: with up to 4 query rows per KV head two fp16 parts, the
        second times 2^11: off by 2^-22 of itself, or by 2^-36 under a power of
        two that puts T at 2^6 at the least, 2^-42 T; a code counts 15 at most:
        15 (2^-22 S + n 2^-42 T).  With more rows one part, off by 2^-11 of itself
        or 2^-31 T, which is given back at the middle code: 7.5 (2^-11 S + n
        2^-31 T).
      - the exponential (2^-22), again where pieces are joined, and products in
        fp32: together 2^-19 A.
      - a logit c (s (q . u) + lo sum(q)): sums and products as in
        kv4_ref.attend for this token's own s and lo, the difference to the
        maximum in force then (which no logit so far beats by more than 6, and
        is no further from 0 than this logit and the largest): d_t = (15 |s| +
        |lo|) (2 (D + 8) 2^-24 c sum|q| + c sum|e|) + 2^-22 (2 |x_t| + max|x| + 6).
        A weight off by e^(+-d_t) moves the output by w_t expm1(d_t) |v_t - out|
        of the sum of such weights, |v_t - out| <= |s_t| u_t + |lo_t| + A.
      - sums in fp32: a matrix unit adds 16 products and may cut each, and the
        sum, at 2^-24; a lane adds 4 of 32 tokens, each sum off by 2^-24; 32 more
        for lanes, warps and pieces: f = 1.1 (n + 32) 2^-24 of A for the codes and
        lows together and of A again for the sum of weights.  With more than
        4 rows the sums that are given back: 15 f S.
    """
    QL, H, D = q.shape
    Hk = k_pool.shape[1]
    g = H // Hk
    split = g * q_len <= 4
    out = torch.zeros((QL, H, D), dtype=torch.float64, device=q.device)
    slack = torch.zeros_like(out)
    kv, vv = ref.values(k_pool), ref.values(v_pool)
    ke, ve = (ref.pool_views(x)[1].contiguous().view(torch.bfloat16).double() for x in (k_pool, v_pool))
    codes = ref.pool_views(v_pool)[0]
    codes = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    for j in range(QL):
        p = n - QL + j
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < lo:
            continue
        at = torch.arange(lo, p + 1, device=q.device)
        b, o = table[at // 16].long(), at % 16
        K, V, U = kv[b, :, o], vv[b, :, o], codes[b, :, o]
        qq = q[j].double().reshape(Hk, g, D)
        x = torch.einsum("hgd,thd->hgt", qq, K) * scale
        w = torch.softmax(x, -1)
        want = torch.einsum("hgt,thd->hgd", w, V)
        s, low = ve[b, :, o, 0].abs(), ve[b, :, o, 1].abs()                     # [n, Hk]
        size = U * s[..., None] + low[..., None]                               # [n, Hk, D]
        ws = w * s.t()[:, None]
        T, S, A = ws.amax(-1)[..., None], ws.sum(-1)[..., None], torch.einsum("hgt,thd->hgd", w, size)
        m = len(at)
        f = 1.1 * (m + 32) * 2.0 ** -24
        e = 15 * (2.0 ** -22 * S + m * 2.0 ** -42 * T) if split else 7.5 * (2.0 ** -11 * S + m * 2.0 ** -31 * T) + 15 * f * S
        sk, lk = ke[b, :, o, 0].abs().t()[:, None], ke[b, :, o, 1].abs().t()[:, None]
        qs = qq.abs().sum(-1, keepdim=True) * abs(scale)
        lost = (qq - ref.query_integers(qq)).abs().sum(-1, keepdim=True) * abs(scale)
        d = (15 * sk + lk) * (2 * (D + 8) * 2.0 ** -24 * qs + lost) + 2.0 ** -22 * (2 * x.abs() + x.amax(-1, keepdim=True).abs() + 6)
        moved = w * torch.expm1(d)
        share = moved.sum(-1)[..., None]
        e = e + (torch.einsum("hgt,thd->hgd", moved, size) + share * A) / (1 - share) + (2.0 ** -19 + 2 * f) * A
        out[j], slack[j] = want.reshape(H, D), e.expand(Hk, g, D).reshape(H, D)
    return out, slack


def pools(gen, n, Hk, D):
    """Pools of one sequence's blocks in order, K rows constant (scale 0, low
    0: a logit is low sum(q)), V rows of random codes under scale 1, low -7.5."""
    NB = -(-n // 16)
    k, v = (torch.randint(0, 256, (NB, Hk, 8 * D + 64), generator=gen, device="cuda", dtype=torch.uint8) for _ in range(2))
    set_rows(k, torch.zeros(NB * 16), torch.zeros(NB * 16))
    set_rows(v, torch.ones(NB * 16), torch.full((NB * 16,), -7.5))
    return k, v


def set_rows(pool, scale, low):
    """Every KV head's rows take these scales and lows [NB * 16], rounded to bf16."""
    NB, Hk = pool.shape[:2]
    e = torch.stack((scale, low), -1).to(torch.bfloat16).cuda().view(NB, 1, 16, 2).expand(NB, Hk, 16, 2).contiguous()
    ref.pool_views(pool)[1].copy_(e.view(torch.uint8).view(NB, Hk, 16, 4))
