"""What the calls on paged caches make of wrong arguments, on the host."""
import ctypes as ct
import math

import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged
from tests.test_quant_cache import fake_attention, fake_format, fake_pages, fake_rows, quant_pages


def test_an_object_of_another_type_is_refused_before_the_call():
    """A structure of another type, an address, bytes of another length: an exception, not a call on a wrong address."""
    L, n = C.lib(), ct.c_size_t()
    plain, p, f, a, r = fake_pages(C=64, token_stride=64), quant_pages(), fake_format(), fake_attention(), fake_rows()
    ref = ct.byref
    assert L.cg_attend_ws_bytes(ref(plain), ref(a), ref(n)) == C.CG_OK
    assert L.cg_attend_ws_bytes(ref(plain), bytes(a), ref(n)) == C.CG_OK
    assert L.cg_attend_ws_bytes(ref(plain), None, ref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend_ws_bytes(ref(p), ref(f), bytes(a), ref(n)) == C.CG_OK
    assert L.cg_quant_write(ref(p), ref(f), bytes(fake_rows(n_rows=0)), 0, None) == C.CG_OK
    for wrong in (ref(r), ref(f), ct.addressof(a), bytes(a)[:-4], bytes(r), bytearray(bytes(a)), "a", 0):
        with pytest.raises(ct.ArgumentError):
            L.cg_attend_ws_bytes(ref(plain), wrong, ref(n))
        with pytest.raises(ct.ArgumentError):
            L.cg_attend(ref(plain), wrong, 4096, 1 << 30, 0, None)
        with pytest.raises(ct.ArgumentError):
            L.cg_quant_attend_ws_bytes(ref(p), ref(f), wrong, ref(n))
        with pytest.raises(ct.ArgumentError):
            L.cg_quant_attend(ref(p), ref(f), wrong, 4096, 1 << 30, 0, None)
    for call in (L.cg_quant_write, L.cg_quant_read):
        for args in ((ref(f), ref(f), ref(r)), (ref(p), ref(p), ref(r)), (ref(p), ref(f), ref(a)), (ref(p), ref(f), bytes(r) + b"0"),
                     (ct.addressof(p), ref(f), ref(r)), (ref(p), ct.addressof(f), ref(r)), (ref(p), ref(f), ct.addressof(r))):
            with pytest.raises(ct.ArgumentError):
                call(*args, 0, None)


def host_caches():
    i32 = dict(dtype=torch.int32)
    state = lambda: (torch.zeros((3, 4), **i32), torch.zeros(3, **i32), torch.zeros(5, **i32), torch.zeros(1, **i32))  # noqa: E731
    return (paged.PagedCache(torch.zeros((2, 5, 2, 16, 64), dtype=torch.float16), *state()),
            paged.QuantCache(torch.zeros((2, 5, 2, 16, 24), dtype=torch.int16), *state(), n_kv_heads=1, head_dim=64))


@pytest.mark.parametrize("kw", [dict(scale=1e39), dict(scale=-1e300), dict(scale=math.inf), dict(scale=math.nan), dict(layer=1 << 32),
                                dict(layer=2), dict(shared_blocks=1 << 32), dict(shared_blocks=5), dict(shared_blocks=1, shared_slot=1 << 40)])
def test_numbers_that_their_type_cannot_hold_are_invalid_arguments(kw):
    """As those that the library refuses: neither wrapped into range nor an exception of another kind."""
    q = torch.zeros((2, 1, 4, 64), dtype=torch.float16)
    for cache in host_caches():
        with pytest.raises(C.CodecError) as e:
            cache.attend(kw.get("layer", 0), q, **{k: v for k, v in kw.items() if k != "layer"})
        assert e.value.code == C.CG_ERR_INVALID_ARG
    if "layer" in kw and kw["layer"] > 2:
        x = torch.zeros((1, 3, 64), dtype=torch.float16)
        for call in (lambda: cache.write(x, x, **kw), lambda: cache.read(out=(x, x), **kw)):
            with pytest.raises(C.CodecError) as e:
                call()
            assert e.value.code == C.CG_ERR_INVALID_ARG


def test_a_server_of_many_contexts_keeps_few_sizes(monkeypatch):
    """A quantised cache asks for its workspace by the number of shared blocks; what it remembers of that is bounded."""
    i32 = dict(dtype=torch.int32)
    cache = paged.QuantCache(torch.zeros((1, 5, 2, 16, 24), dtype=torch.int16), torch.zeros((3, 9000), **i32), torch.zeros(3, **i32),
                             torch.zeros(5, **i32), torch.zeros(1, **i32), n_kv_heads=1, head_dim=64)
    given = []
    monkeypatch.setattr(cache, "_stream", lambda stream: 0)
    monkeypatch.setattr(cache, "_workspace", lambda n, stream, handle: given.append(n))
    monkeypatch.setattr(cache, "_attend", lambda a, ws, handle: C.CG_OK)
    q = torch.zeros((300, 1, 4, 64), dtype=torch.float16)[:3]
    for _ in range(2):
        for shared in range(1, 9000, 2):
            cache.attend(0, q, shared_blocks=shared)
        assert len(cache._attn) <= 1024
    assert given[:4500] == given[4500:] and len(given) == 9000
