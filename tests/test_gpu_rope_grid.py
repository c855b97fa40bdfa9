"""Rotations give the same bits however a call's tokens are dealt out: batches
around the sizes where a token's rows change from many CTAs to one, and where
the tokens pass one wave of CTAs, against the same tokens a few at a time."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter,R", [(False, 128), (True, 128), (False, 20)])
@pytest.mark.parametrize("H,Hk,kind", [(32, 32, "fp8"), (32, 8, "int4"), (64, 8, "16"), (40, 8, None)])
def test_dealing_out(H, Hk, kind, inter, R):
    require_gpu()
    from paged_kv_cache_424_b200 import binding as p
    D, dtype = 128, torch.bfloat16
    g = torch.Generator("cuda")
    g.manual_seed(H + R)
    f = p.pa_rope_frequencies(R)[0].cuda()
    for T in (1, 99, 170, 171, 197, 237, 296, 342, 395, 591, 593, 1183, 1184, 1185, 1300):
        qkv = torch.randn((T, H + 2 * Hk, D), generator=g, device="cuda").to(dtype)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        pos = torch.randint(0, 100000, (T,), generator=g, device="cuda")
        NB = T // 16 + 3
        slots = torch.randperm(NB * 16, generator=g, device="cuda")[:T]
        slots = torch.where(torch.rand((T,), generator=g, device="cuda") < 0.1, torch.full_like(slots, -1), slots)
        shape = p.int4_cache_shape(NB, Hk, D) if kind == "int4" else (NB, Hk, 16, D)

        def call(step):
            qo = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
            if kind is None:
                ko = torch.full((T, Hk, D), 7.0, dtype=dtype, device="cuda")
                for i in range(0, T, step):
                    s = slice(i, i + step)
                    p.pa_rope(qo[s], q[s], ko[s], k[s], pos[s], f, interleaved=inter)
                return qo, ko
            pools = [torch.zeros(shape, dtype=dtype if kind == "16" else torch.uint8, device="cuda") for _ in "kv"]
            ks = 0.05 if kind == "fp8" else 1.0
            for i in range(0, T, step):
                s = slice(i, i + step)
                p.pa_rope_and_cache(qo[s], q[s], k[s], v[s], *pools, slots[s], pos[s], f, interleaved=inter, k_scale=ks, v_scale=ks)
            return (qo, *pools)

        for a, b in zip(call(T), call(61)):
            assert torch.equal(a, b), T
    assert p.pa_device_error() == 0
