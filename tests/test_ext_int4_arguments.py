"""pa_decode_ext over a 4-bit K pool refuses what does not go with it before anything is launched, as pa_decode_int4
does (CPU: the device checks and the library call are stood in for)."""
import pytest
import torch


@pytest.fixture
def ext(monkeypatch):
    from paged_kv_cache_424_b200 import build
    build.build()
    from paged_kv_cache_424_b200 import binding as b
    calls = []

    class Lib:
        @staticmethod
        def pa_decode_ext(*args):
            calls.append(args)
            return 0

    monkeypatch.setattr(b, "LIB", Lib)
    monkeypatch.setattr(b, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(b, "_on_device", lambda *ts: None, raising=False)
    monkeypatch.setattr(b, "_stream", lambda stream: 0)

    def call(out=None, v=None, tables=None, lens=None):
        q = torch.zeros((3, 2, 8, 64), dtype=torch.float16)
        k = torch.zeros(b.int4_cache_shape(10, 2, 64), dtype=torch.uint8)
        calls.clear()
        b.pa_decode_ext(torch.zeros_like(q) if out is None else out, q, k, torch.zeros_like(k) if v is None else v,
                        torch.zeros((3, 4), dtype=torch.int32) if tables is None else tables,
                        torch.zeros(3, dtype=torch.int32) if lens is None else lens, 0.125, 2, 40, q_len=2)
        return len(calls)
    return call


def test_accepted(ext):
    assert ext() == 1


@pytest.mark.parametrize("kw", [dict(v=torch.zeros((9, 2, 576), dtype=torch.uint8)),
                                dict(v=torch.zeros((10, 2, 16, 64), dtype=torch.uint8)),
                                dict(v=torch.zeros((10, 2, 576), dtype=torch.int8)),
                                dict(tables=torch.zeros((2, 4), dtype=torch.int32)),
                                dict(lens=torch.zeros(2, dtype=torch.int32)),
                                dict(out=torch.zeros((3, 2, 8, 64), dtype=torch.bfloat16))])
def test_refused(ext, kw):
    with pytest.raises((ValueError, TypeError)):
        ext(**kw)
