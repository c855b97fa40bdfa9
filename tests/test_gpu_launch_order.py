"""Steps in which every input of a decode over a 16-bit or FP8 cache is written
by the kernel right in front of it, layer after layer into the same buffers: a
captured loop gives bit for bit what calls with a synchronisation around each
give."""
import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    from paged_kv_cache_424_b200 import build
    build.build()
    from paged_kv_cache_424_b200 import binding
    assert binding.pa_device_error() == 0, "device error word set before the test"
    yield
    assert binding.pa_device_error() == 0, "a kernel flagged a device error"


@pytest.mark.parametrize("kind", ["16", "fp8"])
@pytest.mark.parametrize("H,Hk,q_len,S,most", [(32, 8, 1, 6, 300), (64, 8, 1, 2, 3000), (16, 4, 4, 40, 200)])
def test_inputs_written_by_the_kernel_in_front(kind, H, Hk, q_len, S, most):
    from paged_kv_cache_424_b200 import binding as p
    g = torch.Generator("cuda")
    g.manual_seed(H + S)
    layers, D, dtype = 16, 128, torch.bfloat16
    f = p.pa_rope_frequencies(D)[0].cuda()
    row = (most + layers * q_len) // 16 + 1
    shape = (S * row, Hk, 16, D)
    if kind == "fp8":
        pools = [torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    else:
        pools = [torch.randn(shape, generator=g, device="cuda").to(dtype) for _ in range(2)]
    ks = vs = 0.03 if kind == "fp8" else 1.0
    news = [torch.randn((layers, S * q_len, h, D), generator=g, device="cuda").to(dtype) for h in (H, Hk, Hk)]
    tables = torch.stack([torch.randperm(S * row, generator=g, device="cuda").int().view(S, row) for _ in range(layers)])
    lens = torch.randint(1, most, (layers, S), generator=g, device="cuda", dtype=torch.int32)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def loop(sync):
        kc, vc = (x.clone() for x in pools)
        q, k, v = (torch.zeros_like(x[0]) for x in news)
        turned, tab, cl = torch.zeros_like(q), torch.zeros_like(tables[0]), torch.zeros_like(lens[0])
        pos, slots = (torch.zeros(S * q_len, dtype=torch.int64, device="cuda") for _ in range(2))
        outs = torch.full((2, layers) + q.shape, float("nan"), dtype=dtype, device="cuda")

        def wait():
            if sync:
                torch.cuda.synchronize()

        def attend(out):
            p.pa_decode_ext(out.view(S, q_len, H, D), turned.view(S, q_len, H, D), kc, vc, tab, cl, 0.09, Hk, most + q_len, q_len, 0, ks, vs, 0, ws)

        def body():
            for i in range(layers):
                at = (lens[i].long()[:, None] + torch.arange(q_len, device="cuda")[None, :])
                for dst, src in ((q, news[0][i]), (k, news[1][i]), (v, news[2][i])):
                    dst.copy_(src)
                pos.copy_(at.flatten())
                slots.copy_((tables[i].gather(1, at // 16).long() * 16 + at % 16).flatten())
                tab.copy_(tables[i])
                cl.copy_(lens[i] + q_len)
                wait()
                p.pa_rope_and_cache(turned, q, k, v, kc, vc, slots, pos, f, k_scale=ks, v_scale=vs)
                wait()
                attend(outs[0, i])
                wait()
                # a rotation alone in front, and lengths that the caller's kernel has just shortened
                p.pa_rope(turned, q, None, None, pos, f, interleaved=True)
                wait()
                attend(outs[1, i])
                wait()
        return body, outs, (kc, vc, q, k, v, turned, tab, cl, pos, slots)

    body, want, _keep = loop(True)
    body()
    assert bool(want.isfinite().all())
    body, got, _keep2 = loop(False)
    body()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    body, got, _keep3 = loop(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for pool, first in zip(_keep3[:2], pools):
        pool.copy_(first)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
