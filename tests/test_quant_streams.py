"""Calls on a quantised cache from a stream of their own, beside work on the current one, and two caches at once."""
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged, synth
from tests.test_quant_cache import BF16, FP16, _ints, attend, gpu, make


def busy(seconds=0.02):
    """Work on the current stream, and memory of its that is freed while it runs."""
    torch.cuda._sleep(int(seconds * 1.9e9))
    x = torch.full((64 << 20,), 7, dtype=torch.uint8, device="cuda")
    del x


@gpu
def test_a_context_decoded_on_another_stream():
    L, T, Hkv, D, bt = 3, 333, 2, 64, 16
    cfg = C.Config(L, T, Hkv * D)
    enc = C.encode(cfg, synth.ar1_kv(L, T, Hkv * D, 0.95, 2, 0, device="cuda"))
    caches = [paged.QuantCache.empty(L, 30, bt, Hkv, D, 2, 25) for _ in range(2)]
    for cache in caches:
        cache.fork(_ints([-1]), _ints([0]), _ints([T]))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        busy()
        caches[0].decode(cfg, enc, 0, stream=s)
        back = caches[0].read(n_layers=L, rows=T, slots=_ints([0]), stream=s)
        busy()
        s.synchronize()
        caches[1].decode(cfg, enc, 0)
        want = caches[1].read(n_layers=L, rows=T, slots=_ints([0]))
        assert torch.equal(caches[0].pool, caches[1].pool) and all(torch.equal(a, b) for a, b in zip(back, want))
        assert caches[0].lens.tolist() == [T, 0]
        s.wait_stream(torch.cuda.current_stream())
        caches[0].pool[:, :, :, :, :8] = 0
        torch.cuda.synchronize()
    for cache in caches:
        cache.check()


@gpu
@pytest.mark.parametrize("R", [6, 200])
def test_two_caches_on_two_streams_at_once(R):
    """Each has its own workspace; a call's outputs and the next call's belong to its stream."""
    shared, Hkv = 64, 8
    both = [make([shared * 16 + 1 + (r * 131 + 7 * i) % 300 for r in range(R)], shared, 16, Hkv, 64, dtype=t, seed=i)
            for i, t in enumerate((FP16, BF16))]
    streams = [torch.cuda.Stream() for _ in both]
    want = [attend(cache, slots, shared_blocks=shared, seed=5) for cache, slots in both]
    torch.cuda.synchronize()
    outs = [[], []]
    busy()
    for _ in range(6):
        for (cache, slots), s, (q, _, _), o in zip(both, streams, want, outs):
            o.append(cache.attend(1, q, slots=slots, shared_blocks=shared, stream=s))
    torch.cuda.synchronize()
    for (cache, slots), (q, out, lse), o in zip(both, want, outs):
        assert all(torch.equal(x, out) for x in o)
        cache.check()
