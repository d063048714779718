"""The one-shot codec calls on a stream other than the current one."""
import types

import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import synth

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


@pytest.mark.gpu
@needs_gpu
def test_codec_calls_on_another_stream_beside_pending_work():
    """The one-shot codec calls take their buffers on the current stream: what
    is queued there comes first, on whatever stream the call runs."""
    cfg = C.Config(2, 700, 64)
    kv = synth.ar1_kv(2, 700, 64, 0.95, 1, seed=3).cuda()
    enc = C.encode(cfg, kv)
    want, bits = C.decode(cfg, enc), C.ablation(cfg, kv)
    levels = [e for _, e in C.encode_levels(cfg, kv, [1.0, 2.0])]
    s = torch.cuda.Stream()

    def pending():
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for n in (want.numel() * 2, 1, 1 << 12, 1 << 16, 1 << 20, 4 << 20):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)

    def same(a, b):
        return all(torch.equal(getattr(a, f), getattr(b, f)) for f in ("anchors", "scales", "tables", "payload", "stream_off"))

    torch.cuda.synchronize()
    for _ in range(3):
        pending()
        assert torch.equal(C.decode(cfg, enc, stream=s).view(torch.int16), want.view(torch.int16))
        pending()
        assert same(C.encode(cfg, kv, stream=s), enc)
        pending()
        assert all(same(e, f) for (_, e), f in zip(C.encode_levels(cfg, kv, [1.0, 2.0], stream=s), levels))
        pending()
        again = C.ablation(cfg, kv, stream=s)
        for f in C.ABLATION_FIELDS:  # sums of at most `values` positive fp64 terms, in any order
            assert abs(again[f] - bits[f]) <= 2 * bits["values"] * 2.0 ** -53 * bits[f], f


def test_a_codec_call_waits_for_the_stream_its_buffers_are_from(monkeypatch):
    order = []
    s = types.SimpleNamespace(cuda_stream=7, wait_stream=lambda other: order.append(("wait", other)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: order.append("synchronize"))
    monkeypatch.setattr(C, "cg_decode", lambda cfg, enc, out, status, stream: order.append(("decode", stream)))
    enc = types.SimpleNamespace(payload=torch.zeros(1, dtype=torch.uint8))
    C.decode(C.Config(1, 20, 16), enc, stream=s)
    assert order == [("wait", "current"), ("decode", s), "synchronize"]
    order.clear()
    C.decode(C.Config(1, 20, 16), enc)
    assert order == [("decode", None), "synchronize"]
