"""What the calls on paged caches make of wrong arguments, on the host."""
import ctypes as ct

import pytest

from kv_cache_compression_decode_gb300 import codec as C
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
