"""Attention of a cache in 4 or 8 bits by the way that its shared blocks go: through 16-bit values in the workspace, or
against the codes.  Each test says which way it means, and checks that its calls go there."""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged
from tests.test_quant_cache import BF16, FP16, _ints, attend, check, gpu, make, parts, rows_like


def workspace_bytes(fmt, bt, R, nq, Hq, shared):
    """cg_quant_attend_ws_bytes of a made-up pool of this format."""
    words, n = ct.c_uint32(), ct.c_size_t()
    assert C.lib().cg_quant_row(ct.byref(fmt), ct.byref(words)) == C.CG_OK
    row = words.value
    p = C.cg_pages(1 << 30, 1, row, 64, bt, 64 * 2 * bt * row, bt * row, 2 * bt * row, row, 1 << 20, 1 << 21, 1 << 22, 1 << 20, 1 << 20)
    D = fmt.head_dim
    a = C.cg_attention(1 << 32, 1 << 33, None, None, fmt.dtype, R, nq, Hq, fmt.n_kv_heads, D, 0, 0, shared,
                       (ct.c_uint64 * 3)(nq * Hq * D, Hq * D, D), (ct.c_uint64 * 3)(nq * Hq * D, Hq * D, D), 1.0)
    assert C.lib().cg_quant_attend_ws_bytes(ct.byref(p), ct.byref(fmt), ct.byref(a), ct.byref(n)) == C.CG_OK
    return n.value


def through_workspace(fmt, bt, R, nq, Hq, shared):
    """Whether the workspace grows with the shared blocks by their 16-bit values (K, V, and bf16's second part of K)."""
    if not shared:
        return False
    a, b = (workspace_bytes(fmt, bt, R, nq, Hq, s) for s in (shared, shared + 1))
    block = bt * fmt.n_kv_heads * fmt.head_dim * 2 * (3 if fmt.dtype == C.CG_BF16 else 2)
    return b - a == block and a > shared * block


def goes(cache, q, shared, through):
    R, nq, Hq, _ = q.shape
    assert through_workspace(cache._format, cache.block_tokens, R, nq, Hq, shared) == through


@pytest.mark.parametrize("dtype,Hkv,g,R,nq,tokens,through", [
    (C.CG_FP16, 8, 1, 64, 1, 32768, False), (C.CG_BF16, 8, 8, 8, 1, 32768, False),  # 64 rows: eight ranges
    (C.CG_FP16, 8, 1, 72, 1, 16384, True), (C.CG_FP16, 8, 8, 9, 1, 16384, True),    # nine ranges of eight rows
    (C.CG_BF16, 8, 4, 20, 4, 32768, True),                                          # twenty ranges of sixteen
    (C.CG_FP16, 8, 4, 5, 4, 32768, False), (C.CG_FP16, 8, 3, 9, 3, 1 << 20, True),  # five of sixteen; six of sixteen, 81 rows
    (C.CG_FP16, 1, 8, 16, 1, 9984, False), (C.CG_FP16, 1, 8, 16, 1, 10016, True),   # sixteen ranges: 16 more half ranges than 16, times tokens, against 160000
    (C.CG_FP16, 8, 8, 128, 1, 64, False), (C.CG_FP16, 8, 8, 128, 1, 128, True)])
def test_which_way_the_shared_blocks_go(dtype, Hkv, g, R, nq, tokens, through):
    fmt = C.cg_quant(dtype, 4, 128, Hkv, 128)
    assert through_workspace(fmt, 32, R, nq, Hkv * g, tokens // 32) == through


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits,D,group,Hkv,nq,g,bt,shared", [
    (4, 128, 128, 8, 1, 1, 16, 160), (4, 128, 32, 4, 2, 2, 8, 130), (8, 64, 64, 8, 1, 2, 64, 20), (4, 64, 32, 3, 3, 3, 256, 4),
    (8, 128, 64, 6, 1, 1, 32, 110)])
@pytest.mark.parametrize("layout", ["plain", "block_major", "padded"])
def test_pools_heads_and_strides_through_the_workspace(dtype, bits, D, group, Hkv, nq, g, bt, shared, layout):
    """One tile of 128 rows and several; q a slice of a wider tensor, out transposed, slots in another order, a negative scale."""
    R, P = 90, shared * bt
    lens = [P + nq - 1 + (11 * r) % 130 for r in range(R)]
    lens[7] = 0
    cache, slots = make(lens, shared, bt, Hkv, D, bits, group, dtype, layout=layout, seed=shared)
    slots = slots.flip(0).contiguous()
    both = torch.randn((R, nq, Hkv * g, 2, D), generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(dtype)
    q, out = both[:, :, :, 1], torch.zeros((nq, R, Hkv * g, D), dtype=dtype, device="cuda").transpose(0, 1)
    goes(cache, q, shared, True)
    q, out, lse = attend(cache, slots, q=q, out=out, shared_blocks=shared, scale=-0.2)
    cache.check()
    check(cache, q, out, lse, slots, 1, np.float32(-0.2).item(), shared)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("D,g,R", [(64, 1, 128), (64, 2, 52), (128, 1, 81), (64, 1, 129)])
def test_one_tile_of_rows_and_one_more(dtype, D, g, R):
    """Up to 128 rows the two streams of products take the even and the odd tiles of tokens of one tile of rows."""
    shared, bt, Hkv = 110, 32, 8
    cache, slots = make([shared * bt + 1 + r % 3 for r in range(R)], shared, bt, Hkv, D, 4, 64, dtype, seed=R)
    q, out, lse = attend(cache, slots, Hq=Hkv * g, shared_blocks=shared)
    goes(cache, q, shared, True)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5, shared)


@gpu
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (0.0, 1e-30), (1e-20, 1.0), (3.0, 1.0), (-3.0, 1.0), (1e-30, 1e-30)])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_scales_through_the_workspace(dtype, scale, size):
    shared, R = 84, 40
    lens = [shared * 16 + 1 + 37 * r % 90 for r in range(R)]
    cache, slots = make(lens, shared, 16, 2, 64, dtype=dtype)
    q = (rows_like((R, 2, 8, 64), dtype).float() * size).to(dtype)
    goes(cache, q, shared, True)
    q, out, lse = attend(cache, slots, nq=2, q=q, scale=scale, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, np.float32(scale).item(), shared)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_a_prompt_through_the_workspace(dtype):
    shared = 30
    cache, slots = make([480 + 400, 480 + 333], shared, 16, 2, 128, dtype=dtype)
    q, out, lse = attend(cache, slots, nq=333, Hq=4, shared_blocks=shared)
    goes(cache, q, shared, True)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5, shared)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_a_graph_of_the_workspace_replays_with_new_tokens(dtype):
    """A captured decode step is replayed as the sequences grow and as the shared tokens change; eager calls give the same bits."""
    shared, bt, R, Hkv = 50, 16, 200, 8
    lens = [shared * bt + 1 + r % 7 for r in range(R)]
    cache, slots = make([n + 30 for n in lens], shared, bt, Hkv, 64, group=32, dtype=dtype)
    cache.lens[1: R + 1] = _ints(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    k, v, q = (torch.zeros(s, dtype=dtype, device="cuda") for s in ((1, R, Hkv * 64), (1, R, Hkv * 64), (R, 1, Hkv, 64)))
    goes(cache, q, shared, True)
    out, lse = torch.empty_like(q), torch.empty((R, 1, Hkv), device="cuda")
    step = lambda: (cache.write(k, v, layer=1, slots=slots),  # noqa: E731
                    cache.attend(1, q, slots=slots, shared_blocks=shared, out=out, lse=lse))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        cache.lens[slots.long()] += 1
        if n:
            cache.write(rows_like((1, shared * bt, Hkv * 64), dtype, n), rows_like((1, shared * bt, Hkv * 64), dtype, 50 + n), layer=1,
                        slots=_ints([0]))
        graph.replay()
        torch.cuda.synchronize()
        check(cache, q, out, lse, slots, 1, 0.125, shared)
        _, o, e = attend(cache, slots, q=q, shared_blocks=shared, scale=0.125)
        assert torch.equal(o, out) and torch.equal(e, lse)
    cache.check()


@gpu
@pytest.mark.parametrize("R", [4, 200])
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_a_shared_block_outside_the_pool_counts_as_zeros(dtype, R):
    """Flagged, and the others' answers are those of a pool with a block of zeros there; requests that do not see the shared
    blocks are flagged and answered as empty."""
    shared, bt, Hkv = 50, 16, 8
    cache, slots = make([shared * bt + 20 + r % 9 for r in range(R)], shared, bt, Hkv, 64, dtype=dtype)
    q, good, _ = attend(cache, slots, shared_blocks=shared)
    goes(cache, q, shared, R == 200)
    cache.check()
    was = int(cache.tables[0, 7])
    spare = next(b for b in range(cache.pool.shape[1]) if not (cache.tables == b).any())
    cache.pool[:, spare] = 0
    cache.tables[0, 7] = spare
    _, want, want_lse = attend(cache, slots, q=q, shared_blocks=shared)
    cache.check()
    assert not torch.equal(want, good)
    for bad in (4000, -1, 2 ** 31 - 1):
        cache.tables[0, 7] = bad
        _, out, lse = attend(cache, slots, q=q, shared_blocks=shared)
        with pytest.raises(C.CodecError) as e:
            cache.check()
        assert e.value.code == C.CG_ERR_RANGE
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    cache.tables[0, 7] = was
    cache.lens[2] = shared * bt - 1
    _, out, lse = attend(cache, slots, q=q, shared_blocks=shared)
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE and (out[1] == 0).all() and (lse[1] == -math.inf).all()
    keep = [r for r in range(R) if r != 1]
    assert torch.equal(out[keep], good[keep])


@gpu
def test_shared_blocks_past_32_bits_through_the_workspace():
    bt, Hkv, D, R, shared = 256, 32, 128, 72, 10
    row = paged.QuantCache.row_width(Hkv, D)
    n_pool = (1 << 32) // (2 * bt * row) + 20
    pool = torch.empty((1, n_pool, 2, bt, row), dtype=torch.int16, device="cuda")
    table = torch.full((R + 1, shared + 2), -1, dtype=torch.int32)
    table[:, :shared] = n_pool - 1 - torch.arange(shared)
    table[1:, shared] = n_pool - 12
    cache = paged.QuantCache(pool, table.cuda(), _ints([shared * bt] + [shared * bt + 40] * R),
                             torch.ones(n_pool, dtype=torch.int32, device="cuda"), n_kv_heads=Hkv, head_dim=D)
    assert (n_pool - shared) * 2 * bt * row > 1 << 32
    k, v = rows_like((1, shared * bt, Hkv * D), FP16), rows_like((1, shared * bt, Hkv * D), FP16, 1)
    cache.write(k, v, slots=_ints([0]))
    cache.write(k[:, :40], v[:, :40], slots=_ints([1]))
    q, out, lse = attend(cache, _ints(range(1, R + 1)), Hq=Hkv, layer=0, shared_blocks=shared)
    goes(cache, q, shared, True)
    cache.check()
    first = n_pool - 12
    small = paged.QuantCache(cache.pool[:, first:].clone(), torch.where(cache.tables < 0, -1, cache.tables - first), cache.lens,
                             cache.refs[first:].contiguous(), n_kv_heads=Hkv, head_dim=D)
    check(small, q, out, lse, _ints(range(1, R + 1)), 0, D ** -0.5, shared)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits,D,group,Hkv,nq,g,shared", [
    (4, 128, 128, 2, 1, 8, 70), (4, 128, 32, 2, 3, 7, 40), (8, 64, 64, 1, 5, 40, 8), (8, 128, 128, 4, 1, 1, 9), (4, 64, 32, 3, 2, 3, 20)])
def test_many_query_rows_against_the_codes(dtype, bits, D, group, Hkv, nq, g, shared):
    """More than 64 rows, but few shared tokens: the values are those of the codes, without the workspace's rounding."""
    R, bt = 33, 16
    if nq * g < 2:
        R = 80
    lens = [shared * bt + nq - 1 + (13 * r) % 70 for r in range(R)]
    cache, slots = make(lens, shared, bt, Hkv, D, bits, group, dtype, seed=shared)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hkv * g, shared_blocks=shared)
    assert R * nq * g > 64
    goes(cache, q, shared, False)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)  # the tolerance of own tokens


@gpu
@pytest.mark.parametrize("Hkv,shared,through", [(1, 0, False), (1, 6, False), (8, 6, True)])
def test_more_requests_than_a_block_keeps(Hkv, shared, through):
    """More requests than a block's shared memory has lengths for."""
    lens = [shared * 16 + 1 + (r * 7) % 40 if r % 40 else 0 for r in range(1100)]
    cache, slots = make(lens, shared, 16, Hkv, 64)
    q, out, lse = attend(cache, slots, Hq=2 * Hkv, shared_blocks=shared)
    goes(cache, q, shared, through)
    cache.check()
    check(cache, q, out, lse, slots, 1, 0.125, shared if through else 0)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("R", [24, 200])
def test_the_same_bits_again_whatever_ran_before(dtype, R):
    """After another shape has used the workspace, and with anything left in it."""
    shared, Hkv = 64, 8
    lens = [shared * 16 + 1 + (r * 131) % 900 for r in range(R)]
    cache, slots = make(lens, shared, 16, Hkv, 128, group=32, dtype=dtype)
    q, out, lse = attend(cache, slots, shared_blocks=shared)
    goes(cache, q, shared, R == 200)
    for _ in range(3):
        attend(cache, slots[:5].contiguous(), nq=3, Hq=16, seed=8)
        cache._ws.fill_(255)
        _, o, e = attend(cache, slots, q=q, shared_blocks=shared)
        assert torch.equal(o, out) and torch.equal(e, lse)
    cache.check()
