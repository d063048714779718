"""cg_attend against the softmax formula in 64 bits.

Tolerances, derived per element from the inputs (u = half a step of the
16-bit type, w the softmax weights, A = sum_t w_t |V_t|, n tokens):
  * a score is a sum of D products, exact in fp32, added in fp32 in some
    order with at most two units of truncation a step: off by at most
    es = scale * D * 2^-22 * max_t sum_d |q_d K_td|; a weight is then off by a
    factor of at most 1 + 2 es;
  * a weight is rounded to the 16-bit type once (u), and below that type's
    normal range by at most 2^-25 of the largest weight;
  * sums of n terms and the joins of pieces in fp32: n * 2^-23;
  * the result is rounded once: u |out|.
"""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged
from tests.test_paged_pages import fake_pages

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
FP16, BF16 = torch.float16, torch.bfloat16


def _ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def make(lens, shared_blocks=0, bt=16, Hkv=2, D=128, dtype=FP16, layout="plain", L=2, seed=0, slots=None, spare=9):
    """A cache whose slot 0 is the shared context and whose further slots are
    the requests (lens: tokens of each, shared ones included).  Rows of the
    pool that belong to no token hold NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    P, Cc, n_slots = shared_blocks * bt, Hkv * D, len(lens) + 3
    need = [max(0, -(-(n - P) // bt)) if n else 0 for n in lens]
    n_pool = shared_blocks + sum(need) + spare
    ids = np.random.default_rng(seed).permutation(n_pool).tolist()
    width = shared_blocks + max(need + [0]) + 2
    table = np.full((n_slots, width), -1, np.int32)
    order = slots if slots is not None else list(range(1, len(lens) + 1))
    table[0, :shared_blocks] = ids[:shared_blocks]
    at = shared_blocks
    shape = dict(plain=(L, n_pool, 2, bt, Cc), block_major=(n_pool, L, 2, bt, Cc), padded=(L, n_pool, 2, bt, Cc + 24))
    pool = torch.full(shape[layout], float("nan"), dtype=dtype, device="cuda")
    pool = pool.transpose(0, 1) if layout == "block_major" else pool[..., :Cc]
    x = torch.randn((L, n_pool, 2, bt, Cc), generator=g, device="cuda") * torch.exp(
        0.5 * torch.randn(Cc, generator=g, device="cuda"))
    pool[:, ids[:shared_blocks]] = x[:, ids[:shared_blocks]].to(dtype)
    for s, n, k in zip(order, lens, need):
        table[s, :shared_blocks] = ids[:shared_blocks]
        own = ids[at: at + k]
        table[s, shared_blocks: shared_blocks + k] = own
        at += k
        for j, b in enumerate(own):
            rows = min(bt, n - P - j * bt)
            pool[:, b, :, :rows] = x[:, b, :, :rows].to(dtype)
    all_lens = np.zeros(n_slots, np.int32)
    all_lens[0] = P
    all_lens[order] = lens
    cache = paged.PagedCache(pool, _ints(table.reshape(-1)).view(table.shape), _ints(all_lens),
                             torch.ones(n_pool, dtype=torch.int32, device="cuda"))
    return cache, _ints(order)


def check(cache, q, out, lse, slots, layer, scale):
    tables, lens = cache.tables.cpu().numpy(), cache.lens.cpu().numpy()
    R, nq, Hq, D = q.shape
    bt, Hkv = cache.block_tokens, cache.pool.shape[4] // D
    g, u = Hq // Hkv, torch.finfo(q.dtype).eps / 2
    kv, qd = cache.pool[layer].double(), q.double()
    for r, s in enumerate(slots.tolist()):
        n = int(lens[s])
        rows = kv[_ints(tables[s][: -(-n // bt)]).long()].permute(1, 0, 2, 3).reshape(2, -1, Hkv, D)[:, :n]
        for i in range(nq):
            seen = n - nq + 1 + i
            if seen <= 0:
                assert (out[r, i] == 0).all() and (lse[r, i] == -math.inf).all(), (r, i)
                continue
            K, V = rows[0, :seen].repeat_interleave(g, 1), rows[1, :seen].repeat_interleave(g, 1)
            x = torch.einsum("hd,thd->ht", qd[r, i], K) * scale
            es = (torch.einsum("hd,thd->ht", qd[r, i].abs(), K.abs()).amax(1) * abs(scale) * D * 2.0 ** -22)[:, None]
            w = torch.softmax(x, 1)
            ref, A = torch.einsum("ht,thd->hd", w, V), torch.einsum("ht,thd->hd", w, V.abs())
            tiny = seen * 2.0 ** -25 * w.amax(1)[:, None] * V.abs().amax(0)
            tol = u * ref.abs() + (u + 2 * es + seen * 2.0 ** -23 + 2.0 ** -20) * A + tiny + 2.0 ** -25
            err = (out[r, i].double() - ref).abs()
            assert (err <= tol).all(), (r, i, float((err / tol).max()))
            want = torch.logsumexp(x, 1)
            tol = es[:, 0] + (seen + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -22
            assert ((lse[r, i].double() - want).abs() <= tol).all(), (r, i)


def attend(cache, slots, nq=1, Hq=8, D=128, layer=1, scale=None, shared_blocks=0, seed=3, q=None, out=None, **kw):
    R = slots.shape[0]
    if q is None:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        q = (1.5 * torch.randn((R, nq, Hq, D), generator=g, device="cuda")).to(cache.pool.dtype)
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    if out is None:
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    cache.attend(layer, q, slots=slots, shared_slot=0, shared_blocks=shared_blocks, scale=scale, out=out, lse=lse, **kw)
    return q, out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("D,Hq,Hkv,nq", [(128, 8, 2, 1), (64, 2, 2, 1), (128, 14, 2, 3), (64, 40, 1, 5), (128, 3, 3, 2)])
@pytest.mark.parametrize("bt", [8, 16, 64, 256])
def test_own_tokens_only(dtype, D, Hq, Hkv, nq, bt):
    cache, slots = make(LENS, bt=bt, Hkv=Hkv, D=D, dtype=dtype)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, D=D)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("D,Hq,Hkv,nq", [(128, 16, 2, 1), (64, 2, 2, 1), (128, 14, 2, 3), (64, 40, 1, 5)])
@pytest.mark.parametrize("bt,shared", [(8, 1), (16, 70), (64, 5), (256, 3)])
def test_shared_blocks(dtype, D, Hq, Hkv, nq, bt, shared):
    P = shared * bt
    lens = [P + max(n, nq - 1) if n or nq == 1 else 0 for n in LENS if n != 1] + [0, P + nq]
    cache, slots = make(lens, shared, bt, Hkv, D, dtype, seed=shared)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, D=D, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("R", [1, 5, 33, 130])
@pytest.mark.parametrize("nq,Hq,D", [(1, 8, 128), (4, 16, 128), (1, 16, 64)])
def test_batches_over_a_long_context(R, nq, Hq, D):
    """From a few query rows on the shared blocks to many tiles of them; with
    one, several and very unequal own lengths."""
    P, bt = 1500 // 32 * 32, 32
    lens = [P + nq + (37 * r) % 200 for r in range(R)]
    lens[R // 2] = P + 2500
    cache, slots = make(lens, P // bt, bt, 1, D, seed=R)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, D=D, shared_blocks=P // bt)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("Hkv,g,nq", [(4, 8, 1), (8, 8, 4), (12, 1, 1), (6, 5, 2), (32, 1, 1), (4, 3, 7)])
@pytest.mark.parametrize("D,shared", [(128, 0), (128, 9), (64, 0), (64, 9)])
def test_groups_of_heads(Hkv, g, nq, D, shared):
    """Head counts whose heads go four, two and one to a block, on their own
    and behind shared blocks, for few and for many query rows."""
    for R in (2, 30):
        lens = [shared * 16 + (nq + 53 * r % 150 if r % 7 else 0) for r in range(R)]
        lens = [n if n > shared * 16 else 0 for n in lens]
        cache, slots = make(lens, shared, 16, Hkv, D, seed=R)
        q, out, lse = attend(cache, slots, nq=nq, Hq=Hkv * g, D=D, shared_blocks=shared)
        cache.check()
        check(cache, q, out, lse, slots, 1, D ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("shared,Hkv,nq", [(0, 4, 4), (6, 4, 4), (6, 1, 9), (0, 2, 2)])
def test_a_token_reaches_only_the_queries_that_see_it(dtype, shared, Hkv, nq):
    """Infinities and NaNs in K and V of the later drafted tokens: the first
    query's answer is still that of the tokens that it sees."""
    P = shared * 16
    lens = [P + n for n in (nq, nq + 1, 16 + nq // 2, 31 + nq, 100)]
    cache, slots = make(lens, shared, 16, Hkv, 128, dtype)
    q, out, lse = attend(cache, slots, nq=nq, Hq=8 * Hkv // (2 if Hkv > 1 else 1), shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5)
    for j, bad in ((1, math.inf), (nq - 1, math.nan)):  # drafted token j of nq
        for s, n in zip(slots.tolist(), lens):
            at = n - nq + j
            cache.pool[1, cache.tables[s, at // 16].long(), :, at % 16, ::3] = bad
    _, out2, lse2 = attend(cache, slots, q=q, nq=nq, shared_blocks=shared)
    cache.check()
    cache.lens[slots.long()] -= nq - 1  # what the first query sees, as a sequence of its own
    check(cache, q[:, :1], out2[:, :1], lse2[:, :1], slots, 1, 128 ** -0.5)
    assert not torch.isfinite(out2[:, 1:, :, ::3]).any()
    assert not torch.isfinite(lse2[:, 1:]).any()


@pytest.mark.gpu
@needs_gpu
def test_strides_of_single_element_dimensions_are_free():
    """One layer, one block, one query: their strides say nothing."""
    base = torch.randn(4096, device="cuda").to(FP16)
    pool = base[:2 * 8 * 64].as_strided((1, 1, 2, 8, 64), (3, 5, 8 * 64, 64, 1))
    cache = paged.PagedCache(pool, _ints([0]).view(1, 1), _ints([7]), _ints([1]))
    q = base[2048:2048 + 256].as_strided((1, 1, 4, 64), (7, 11, 64, 1))
    out, lse = torch.empty((1, 1, 4, 64), dtype=FP16, device="cuda"), torch.empty((1, 1, 4), device="cuda")
    cache.attend(0, q, out=out, lse=lse)
    cache.check()
    check(cache, q, out, lse, _ints([0]), 0, 64 ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("shared", [0, 6])
def test_more_requests_than_a_block_keeps(shared):
    """More requests than a block's shared memory has lengths for."""
    lens = [shared * 16 + (r * 7) % 40 if r % 40 else 0 for r in range(1100)]
    lens = [n if n > shared * 16 else 0 for n in lens]
    cache, slots = make(lens, shared, 16, 1, 64)
    q, out, lse = attend(cache, slots, Hq=2, D=64, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 64 ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("shared", [0, 6])
def test_more_requests_than_threads(shared):
    rng = np.random.default_rng(5)
    lens = [shared * 16 + int(n) if n else 0 for n in rng.integers(0, 90, 400)]
    cache, slots = make(lens, shared, 16, 1, 64, BF16)
    q, out, lse = attend(cache, slots, Hq=4, D=64, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 64 ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("layout", ["block_major", "padded"])
@pytest.mark.parametrize("shared,R", [(0, 9), (9, 9), (9, 70)])
def test_layouts_strides_slot_order_and_scale(layout, shared, R):
    """Other pool layouts, q as a slice of a fused projection, out in another
    order, slots out of order, a negative scale."""
    lens = [shared * 16 + 1 + 11 * (r % 9) for r in range(R)]
    order = np.random.default_rng(R).permutation(np.arange(1, R + 3))[:R].tolist()
    cache, slots = make(lens, shared, 16, 2, 128, layout=layout, slots=order)
    fused = torch.randn((R, 2, 12, 128), device="cuda").to(FP16)
    out = torch.full((8, R, 2, 128), float("nan"), dtype=FP16, device="cuda").permute(1, 2, 0, 3)
    q, out, lse = attend(cache, slots, q=fused[:, :, 2:10], out=out, shared_blocks=shared, scale=-0.07, layer=0)
    cache.check()
    check(cache, q, out, lse, slots, 0, -0.07)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("R", [3, 40])
@pytest.mark.parametrize("scale", [0.0, 1e-20, 3.0])
def test_scales(R, scale):
    """Scale 0 gives the mean of the values that a query sees."""
    cache, slots = make([9 * 16 + 3 + 7 * r for r in range(R)], 9, 16, 2, 64)
    q, out, lse = attend(cache, slots, nq=2, Hq=8, D=64, scale=scale, shared_blocks=9)
    cache.check()
    check(cache, q, out, lse, slots, 1, scale)


@pytest.mark.gpu
@needs_gpu
def test_default_slots_and_no_lse():
    cache, slots = make([40, 7], bt=16, Hkv=1)
    q = torch.randn((3, 1, 4, 128), device="cuda").to(FP16)  # slots 0 (empty), 1, 2
    out = cache.attend(0, q)
    cache.check()
    lse = torch.empty((3, 1, 4), device="cuda")
    again = cache.attend(0, q, slots=_ints([0, 1, 2]), lse=lse)
    assert torch.equal(out, again) and (out[0] == 0).all()
    check(cache, q, out, lse, _ints([0, 1, 2]), 0, 128 ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("R", [2, 40])
def test_large_scores_and_infinite_values(R):
    """Scores far apart (weights that underflow), keys at the type's largest
    value, and an infinite V that every query sees."""
    shared, bt = 9, 16
    cache, slots = make([shared * bt + 20 + r for r in range(R)], shared, bt, 1, 128, seed=4)
    cache.pool[1, cache.tables[0, 3].long(), 0, 5] *= 300.0
    q, out, lse = attend(cache, slots, Hq=8, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5)
    cache.pool[1, cache.tables[0, 2].long(), 1, 7, 9] = math.inf
    q, out, lse = attend(cache, slots, Hq=8, shared_blocks=shared)
    cache.check()
    # a weight that underflows makes 0 * inf; either way the value is not finite, and only this channel's
    assert not torch.isfinite(out[..., 9]).any()
    out[..., 9] = 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
@needs_gpu
def test_same_bits_every_time_and_for_a_batch_order():
    lens = [9 * 16 + 1 + 50 * r for r in range(24)]
    cache, slots = make(lens, 9, 16, 2, 128)
    q, out, lse = attend(cache, slots, Hq=16, shared_blocks=9)
    for _ in range(3):
        _, o, z = attend(cache, slots, q=q, shared_blocks=9)
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.gpu
@needs_gpu
def test_graph_replays_with_new_lengths_and_another_stream():
    """A captured step reads tables, lengths and q as they are on replay."""
    cache, slots = make([96 + 40, 96 + 64, 96 + 2], 6, 16, 2, 128)
    for s, n in ((1, 96 + 64), (3, 96 + 16)):  # tokens up to the end of the blocks
        blocks = cache.tables[s, 6: -(-n // 16)].long()
        cache.pool[:, blocks] = torch.nan_to_num(cache.pool[:, blocks], nan=0.25)
    q = torch.randn((3, 1, 8, 128), device="cuda").to(FP16)
    out, lse = torch.empty_like(q), torch.empty((3, 1, 8), device="cuda")
    kw = dict(slots=slots, shared_blocks=6, out=out, lse=lse)
    cache.attend(1, q, **kw)  # sizes the workspace
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cache.attend(1, q, **kw)
    for step in range(3):
        q.normal_()
        cache.lens[1:4] += torch.tensor([step, -step, step], dtype=torch.int32, device="cuda")
        out.fill_(float("nan"))
        graph.replay()
        cache.check()
        check(cache, q, out, lse, slots, 1, 128 ** -0.5)
    torch.cuda.synchronize()
    out2 = cache.attend(1, q, slots=slots, shared_blocks=6, stream=s)
    s.synchronize()
    assert torch.equal(out2, out)


@pytest.mark.gpu
@needs_gpu
def test_refused_requests_are_flagged_and_answered_as_empty():
    P = 6 * 16
    for slot, length in ((1, P - 1), (1, 1 << 20), (99, None), (1, P)):
        nq = 3 if length == P else 1  # P tokens with 3 query tokens: the first lies in the shared blocks
        cache, slots = make([P + 10, P + 20], 6, 16, 2, 128)
        if length is not None:
            cache.lens[slot] = length
        else:
            slots[0] = slot
        q, out, lse = attend(cache, slots, nq=nq, shared_blocks=6)
        with pytest.raises(C.CodecError) as e:
            cache.check()
        assert e.value.code == C.CG_ERR_RANGE
        assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
        check(cache, q[1:], out[1:], lse[1:], slots[1:], 1, 128 ** -0.5)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("R", [2, 40])
@pytest.mark.parametrize("bad", [4000, -1, 2 ** 31 - 1])
def test_blocks_outside_the_pool_are_flagged(R, bad):
    cache, slots = make([96 + 20] * R, 6, 16, 2, 128)
    cache.tables[1, 6] = bad
    q, out, lse = attend(cache, slots, shared_blocks=6)
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE
    check(cache, q[1:], out[1:], lse[1:], slots[1:], 1, 128 ** -0.5)
    cache.tables[0, 2] = bad
    attend(cache, slots, q=q, shared_blocks=6)
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("R", [2, 40])
def test_block_offsets_past_32_bits(R):
    bt, n_pool, gap, D = 16, 9, 1 << 30, 128
    flat = torch.empty(8 * gap + 2 * bt * D, dtype=FP16, device="cuda")
    pool = flat.as_strided((1, n_pool, 2, bt, D), (flat.numel() // 8 * 8, gap, bt * D, D, 1))
    pool.copy_(torch.randn((1, n_pool, 2, bt, D), device="cuda"))
    tables = np.full((R + 1, 4), -1, np.int32)
    tables[:, :3] = [8, 0, 6]
    tables[1:, 3] = [1 + r % 5 for r in range(R)]  # the last block: rows that several requests may read
    cache = paged.PagedCache(pool, _ints(tables.reshape(-1)).view(tables.shape), _ints([48] + [64 - r % 9 for r in range(R)]),
                             torch.ones(n_pool, dtype=torch.int32, device="cuda"))
    slots = _ints(range(1, R + 1))
    q, out, lse = attend(cache, slots, Hq=4, layer=0, shared_blocks=3)
    cache.check()
    check(cache, q, out, lse, slots, 0, D ** -0.5)


# ---------------------------------------------------------------------------
# Refusals on the host (no GPU)
# ---------------------------------------------------------------------------

def fake_attention(**kw):
    d = dict(q=1 << 28, out=1 << 29, lse=None, slots=None, dtype=C.CG_FP16, n_requests=4, n_queries=1, n_q_heads=8,
             n_kv_heads=1, head_dim=64, layer=1, shared_slot=0, shared_blocks=2, scale=0.125)
    qs, os_ = kw.pop("q_stride", (512, 512, 64)), kw.pop("out_stride", (512, 512, 64))
    d.update(kw)
    a = C.cg_attention(**d)
    a.q_stride[:], a.out_stride[:] = qs, os_
    return a


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(out=None), dict(q=(1 << 28) + 8), dict(out=(1 << 29) + 2), dict(lse=4098), dict(slots=4097),
    dict(dtype=2), dict(n_requests=0), dict(n_queries=0), dict(n_q_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=2),
    dict(head_dim=32), dict(head_dim=0), dict(layer=2), dict(shared_slot=8), dict(shared_blocks=13),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=(512, 512, 60)), dict(out_stride=(516, 512, 64))])
def test_bad_attention_is_refused_on_the_host(kw):
    L, p, n = C.lib(), fake_pages(), ct.c_size_t()
    assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(fake_attention()), ct.byref(n)) == C.CG_OK
    a = fake_attention(**kw)
    assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(a), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_attend(ct.byref(p), ct.byref(a), 4096, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(pool=None), dict(tables=None), dict(lens=None), dict(pool=(1 << 30) + 8), dict(block_tokens=4), dict(C=96),
    dict(block_tokens=24), dict(layer_stride=100), dict(kv_stride=1020), dict(block_stride=2052), dict(token_stride=68),
    dict(n_slots=0), dict(n_blocks=0), dict(n_blocks=1 << 27), dict(L=0), dict(kv_stride=1 << 40), dict(kv_stride=0),
    dict(block_stride=0)])
def test_bad_pool_is_refused_on_the_host(kw):
    L, a, n = C.lib(), fake_attention(), ct.c_size_t()
    p = fake_pages(**kw)
    assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(a), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_attend(ct.byref(p), ct.byref(a), 4096, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG


def test_workspace_is_checked_on_the_host():
    L, p, a, n = C.lib(), fake_pages(), fake_attention(), ct.c_size_t()
    assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(a), ct.byref(n)) == C.CG_OK
    assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(a), None) == C.CG_ERR_INVALID_ARG
    assert L.cg_attend(ct.byref(p), ct.byref(a), None, n.value, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_attend(ct.byref(p), ct.byref(a), 4096 + 128, n.value, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_attend(ct.byref(p), ct.byref(a), 4096, n.value - 1, 0, None) == C.CG_ERR_RANGE
