"""seq_order over 4-bit caches: with a partition size sequences are scheduled in
it and an entry outside the batch is skipped and flagged; an automatic call checks
and flags it, and computes every sequence."""
import pytest
import torch

import kv4_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,q_len", [(4, 1), (1, 3), (8, 2)])
@pytest.mark.parametrize("P", [0, 16, 64, 4096])
def test_order_and_entries_outside_the_batch(group, q_len, P):
    require_gpu()
    from paged_kv_cache_424_b200 import binding as p
    assert p.pa_device_error() == 0
    g = torch.Generator("cuda")
    g.manual_seed(P + group)
    lens = [5, 900, 0, 130, 17, 400, 1]
    S, Hk, D, row = len(lens), 2, 64, 60
    kc, vc = ref.random_pool(g, S * row, Hk, D), ref.random_pool(g, S * row, Hk, D)
    tables = torch.randperm(S * row, generator=g, device="cuda").int().view(S, row)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = torch.randn((S, q_len, Hk * group, D), generator=g, device="cuda").half()

    def run(order):
        out = torch.full_like(q, 7.0)
        n = p.pa_decode_ext_workspace_size(p.ext_dims(q, kc, tables), p.pa_decode_opts(q_len, 0, 1.0, 1.0), 900, P)
        ws = torch.empty((max(n, 16),), dtype=torch.uint8, device="cuda")
        order = None if order is None else torch.tensor(order, dtype=torch.int32, device="cuda")
        p.pa_decode_ext(out, q, kc, vc, tables, cl, 0.125, Hk, 900, q_len, 0, 1.0, 1.0, P, ws, seq_order=order)
        return out, p.pa_device_error()

    want, word = run(None)
    assert word == 0
    exact, slack = ref.attend(q, kc, vc, tables, cl, 0.125, q_len)
    ref.near(want, exact, slack, "no order")
    got, word = run([6, 1, 3, 0, 5, 4, 2])
    assert word == 0 and torch.equal(got, want)
    for bad in (S, -1):
        got, word = run([6, 1, bad, 0, 5, 4, 2])  # sequence 3 is not listed
        assert word == 2
        for s in range(S):
            if s != 3:
                assert torch.equal(got[s], want[s])
        # a partition size: nothing of it is computed (the merge of several partitions may write what the workspace holds)
        if P == 4096:
            assert bool((got[3] == 7.0).all())
        if P == 0:
            assert torch.equal(got[3], want[3])
