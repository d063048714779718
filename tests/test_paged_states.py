"""Paged caches in states and uses off the usual path: rows with gaps, lost
references, corrupt entries, other streams, reassigned tensors, empty calls."""
import contextlib
import ctypes as ct
import types

import numpy as np
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged
from tests.test_paged_attend import attend, check, fake_attention, make
from tests.test_paged_pages import NB, Model, _cache, _ints, fake_pages

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


def flagged(cache, code):
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == code


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("first", ["lost to a compaction", "lost to a fork"])
def test_a_row_without_its_first_block_is_ended_whole(first):
    """A compaction and a fork write NO_BLOCK over a corrupt first entry; the
    other blocks of that row still lose their references when it ends."""
    cache = _cache()
    cache.fork(_ints([-1]), _ints([0]), _ints([50]))  # blocks 0..3
    cache.lens[0] = 50
    cache.tables[0, 0] = 4000
    cache.refs[0] = 0  # the block that the entry named is nobody's now
    if first == "lost to a compaction":
        cache.compact()  # live: 1, 2, 3 -> block 3 moves to 0
        flagged(cache, C.CG_ERR_CORRUPT)
        assert cache.tables[0].tolist()[:4] == [NB, 1, 2, 0]
        ended = 0
    else:
        cache.fork(_ints([0]), _ints([5]), _ints([0]))
        flagged(cache, C.CG_ERR_CORRUPT)
        assert cache.tables[5, 0].item() == NB and cache.lens[5].item() == 50
        ended = 5
    before = np.bincount([b for b in cache.tables.view(-1).tolist() if 0 <= b < 40], minlength=40)
    assert np.array_equal(cache.refs.cpu().numpy(), before)
    row = [b for b in cache.tables[ended].tolist() if b >= 0]
    cache.free(_ints([ended, ended]))
    cache.check()
    want = before - np.bincount(row, minlength=40)
    assert np.array_equal(cache.refs.cpu().numpy(), want)
    assert (cache.tables[ended] == NB).all() and cache.lens[ended].item() == 0


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("refs", [0, 1, 5, 299])
def test_rows_that_share_lost_references_end_at_zero(refs):
    """300 rows hold the same twelve blocks, which have fewer references than
    that: ended in one call, the counts stop at zero, whatever the order."""
    cache = _cache(slots=300)
    row = _ints(range(7, 19))
    for _ in range(20):
        cache.tables[:] = row
        cache.lens.fill_(12 * 16)
        cache.refs.zero_()
        cache.refs[row.long()] = refs
        cache.free(_ints(range(300)))
        flagged(cache, C.CG_ERR_CORRUPT)
        assert (cache.refs == 0).all() and (cache.tables == NB).all() and (cache.lens == 0).all()


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("slots,width,gap", [(8, 12, 1), (8, 12, 11), (700, 3000, 2999), (700, 3000, 513)])
def test_fork_refuses_a_child_that_holds_any_block(slots, width, gap):
    """A slot of length 0 whose row begins empty and holds a block further on
    is not empty: nothing of the call is done, its siblings' part neither."""
    cache = _cache(n_pool=40, bt=1, Cc=8, slots=slots, width=width)
    cache.fork(_ints([-1]), _ints([0]), _ints([5]))
    cache.lens[0] = 5
    cache.tables[slots - 1, gap] = 30
    cache.refs[30] = 1
    m = Model(cache)
    children = [1, slots - 1] if slots == 8 else list(range(1, slots))
    cache.fork(_ints([0] * len(children)), _ints(children))
    flagged(cache, C.CG_ERR_RANGE)
    m.check(cache)
    cache.free(_ints([slots - 1]))
    m.free([slots - 1])
    cache.fork(_ints([0] * len(children)), _ints(children))  # the next call is not affected
    m.fork([0] * len(children), children, [0] * len(children))
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("bad", [4000, NB])
@pytest.mark.parametrize("n", [5, 50])
def test_fork_of_a_context_whose_last_block_is_corrupt(n, bad):
    """The child has no block where the parent's partly filled one lies outside
    the pool: not one with whatever its last owner left in it."""
    cache = _cache()
    cache.fork(_ints([-1]), _ints([0]), _ints([n]))
    cache.lens[0] = n
    full = n // 16
    cache.tables[0, full] = bad
    m = Model(cache)
    cache.fork(_ints([0, 0]), _ints([3, 4]), _ints([20, 0]))
    flagged(cache, C.CG_ERR_CORRUPT)
    first = full + 1  # fresh blocks are numbered from here: one for each tail (not taken), then the reserve
    more = (n + 20 + 15) // 16 - full - 1
    shared = m.tables[0][:full].tolist()
    for slot, row in ((3, shared + [NB] + list(range(first + 1, first + 1 + more))), (4, shared + [NB])):
        m.tables[slot, : len(row)] = row
        m.lens[slot] = n
        for b in row:
            m.refs[b] += b >= 0
    m.check(cache)
    cache.free(_ints([3, 4]))
    m.free([3, 4])
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_a_fresh_block_that_a_corrupt_parent_names_has_both_references():
    """The parent's row names a free block, which the same call hands out:
    the count is the same in any order, one for each entry of the children."""
    for _ in range(50):
        cache = _cache(n_pool=200, slots=9, width=12)
        cache.fork(_ints([-1]), _ints([0]), _ints([64]))
        cache.lens[0] = 64
        cache.tables[0, 3] = 4  # free; block 3 keeps the reference that the entry had
        cache.fork(_ints([0] * 8), _ints(range(1, 9)), _ints([16] * 8))
        cache.check()
        assert cache.tables[1:, 3].tolist() == [4] * 8 and cache.tables[1:, 4].tolist() == list(range(4, 12))
        assert cache.refs[:12].tolist() == [9, 9, 9, 1, 9] + [1] * 7


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,Hkv,nq,shared", [(128, 4, 1, 0), (64, 1, 3, 0), (128, 2, 1, 100), (64, 4, 1, 4)])
def test_the_small_weights_of_a_long_context_count(dtype, D, Hkv, nq, shared):
    """One token outweighs each of the others by e^18, past the 2^25 below
    which an fp16 weight relative to the largest is zero; together the others
    carry 3% of the output.  There are so many requests that one block takes
    one's tokens alone, that token first.  A weight is rounded once (u), and
    below fp16's normal range, with the largest at 2^15, by at most 2^-40 of
    the largest.  The rest as for the other attention tests."""
    n, bt, big, R = 32768, 16, 18.0, 304
    n_pool = n // bt + 1
    pool = torch.zeros((1, n_pool, 2, bt, Hkv * D), dtype=dtype, device="cuda")
    pool[:, :, 1] = 64.0
    row = np.random.default_rng(0).permutation(n_pool)[: n // bt]
    at = shared * bt + 3  # the token that outweighs the others, among the requests' own
    pool[0, row[at // bt], 0, at % bt, ::D] = big
    pool[0, row[at // bt], 1, at % bt] = 1.0
    tables = _ints(np.tile(row, R)).view(R, -1)
    cache = paged.PagedCache(pool, tables, _ints([n] * R), torch.full((n_pool,), R, dtype=torch.int32, device="cuda"))
    q = torch.zeros((R, nq, Hkv, D), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    lse = torch.empty((R, nq, Hkv), device="cuda")
    out = cache.attend(0, q, shared_slot=0, shared_blocks=shared, scale=1.0, lse=lse)
    cache.check()
    u = torch.finfo(dtype).eps / 2
    es = big * D * 2.0 ** -22
    for i in range(nq):
        seen = n - nq + 1 + i
        z = np.exp(big) + (seen - 1)
        ref = (np.exp(big) * 1.0 + (seen - 1) * 64.0) / z
        tol = u * ref + (u + 2 * es + seen * 2.0 ** -23 + 2.0 ** -20) * ref + seen * 2.0 ** -40 * 64.0 + 2.0 ** -25
        assert (out[:, i].double() - ref).abs().max().item() <= tol
        want = np.log(z)
        assert (lse[:, i].double() - want).abs().max().item() <= es + (seen + 8) * 2.0 ** -23 + want * 2.0 ** -22


@pytest.mark.gpu
@needs_gpu
def test_a_call_on_another_stream_beside_pending_work():
    """Memory that the current stream is still to write, freed and asked for
    again by a call on another stream: the call's results stay its own."""
    cache, slots = make([40, 300, 70], bt=16, Hkv=2)
    q = torch.randn((3, 1, 8, 128), device="cuda").to(torch.float16)
    want = cache.attend(1, q, slots=slots)
    s = torch.cuda.Stream()
    caches = [paged.PagedCache(cache.pool, cache.tables, cache.lens, cache.refs, cache.status) for _ in range(5)]
    torch.cuda.synchronize()
    for fresh in caches:
        torch.cuda._sleep(20_000_000)  # about 10 ms
        dropped = [torch.empty_like(q) for _ in range(8)] + [torch.empty(1 << 22, dtype=torch.uint8, device="cuda")]
        for t in dropped:
            t.fill_(255 if t.dtype == torch.uint8 else float("nan"))
        del dropped, t
        out = fresh.attend(1, q, slots=slots, stream=s)
        s.synchronize()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(out, want)
        cache.check()


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,Hq,Hkv,D,shared", [(33, 4, 4, 128, 0), (65, 2, 1, 64, 6), (150, 4, 2, 128, 6), (500, 1, 1, 128, 0)])
def test_a_prompt_of_many_tokens_over_its_context(dtype, nq, Hq, Hkv, D, shared):
    """The question after a context: each query token sees those before it, row
    ranges begin and end inside the drafted part, one request has no context."""
    P = shared * 16
    lens = [P + nq + 77, P + nq - (shared > 0), 0]
    cache, slots = make(lens, shared, 16, Hkv, D, dtype, seed=nq)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, D=D, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


# ---------------------------------------------------------------------------
# The binding, with the library and the GPU replaced (no GPU)
# ---------------------------------------------------------------------------

def cpu_cache():
    i32 = dict(dtype=torch.int32)
    return paged.PagedCache(torch.zeros((2, 5, 2, 16, 64), dtype=torch.float16), torch.zeros((3, 4), **i32),
                            torch.zeros(3, **i32), torch.zeros(5, **i32))


class FakeLib:
    """Counts the calls that would have launched something."""

    def __init__(self, ws_bytes=1000):
        self.launched, self.ws_bytes = [], ws_bytes

    def cg_attend_ws_bytes(self, pages, attention, n):
        n._obj.value = self.ws_bytes
        return C.CG_OK

    def __getattr__(self, name):
        def call(*args):
            self.launched.append((name, args))
            return C.CG_OK
        return call


def host_cache(monkeypatch, index=0, current=0):
    """A cache of CPU tensors that takes itself for one on GPU `index`."""
    cache = cpu_cache()
    fake = FakeLib()
    monkeypatch.setattr(paged, "lib", lambda: fake)
    monkeypatch.setattr(C, "lib", lambda: fake)
    monkeypatch.setattr(paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(paged, "_current_device", lambda: current, raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
    cache._index = index
    return cache, fake


def test_a_pool_on_another_device_is_refused(monkeypatch):
    """Kernels run on the current device: with the pool on another one nothing is launched."""
    cache, fake = host_cache(monkeypatch, index=1, current=0)
    one = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.float16)
    for call in (lambda: cache.fork(one, one), lambda: cache.free(one), lambda: cache.compact(),
                 lambda: cache.copy(one, one), lambda: cache.attend(0, q),
                 lambda: cache.decode(C.Config(2, 20, 64), None, 0)):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not fake.launched


def test_decode_into_host_memory_is_refused():
    cache = cpu_cache()
    with pytest.raises(ValueError, match="not in GPU memory"):
        cache.decode(C.Config(2, 20, 64), None, 0)


def test_memory_of_a_call_belongs_to_its_stream(monkeypatch):
    """out, remap and the workspace are allocated on the stream whose kernels
    write them, and a workspace that another stream goes on to use is recorded
    there: the allocator then hands none of it out too early."""
    cache, fake = host_cache(monkeypatch)
    at, recorded = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, at[0] = at[0], stream
        yield
        at[0] = before

    empty, where = torch.empty, []

    def logged(*args, **kw):
        where.append(at[0])
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", logged)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    status = cache.status.data_ptr()
    s, r = types.SimpleNamespace(cuda_stream=7), types.SimpleNamespace(cuda_stream=8)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.float16)
    fake.ws_bytes = 1 << 20
    cache.attend(0, q, stream=s)
    assert where == [s, s]  # out and the workspace
    name, args = fake.launched[-1]
    assert name == "cg_attend" and args[-1] == 7
    ws = args[2]
    where.clear()
    recorded.clear()
    cache.attend(0, q, stream=s)
    assert where == [s] and not recorded
    cache.attend(0, q, stream=r)
    cache.attend(0, q, stream=r)
    assert sorted(recorded, key=str) == sorted([(ws, r), (status, r)], key=str)
    cache.attend(0, q)
    assert recorded[2:] == [(ws, "current"), (status, "current")] and where == [s, r, r, None]
    where.clear()
    cache.compact(stream=s)
    assert where == [s]
    cache.compact()
    assert where == [s, None]


def test_check_waits_for_its_own_reset(monkeypatch):
    """After check() the status is zero on the device, not only queued to be:
    an error that a call on another stream finds next is not wiped out."""
    cache = cpu_cache()
    at_sync = []
    monkeypatch.setattr(torch.cuda, "synchronize", lambda device=None: at_sync.append(cache.status.item()))
    cache.status[0] = 1 << C.CG_ERR_RANGE
    flagged(cache, C.CG_ERR_RANGE)
    assert at_sync == [1 << C.CG_ERR_RANGE, 0]
    at_sync.clear()
    cache.check()
    assert set(at_sync) == {0}


@pytest.mark.parametrize("name", ["pool", "tables", "lens", "refs", "status"])
def test_the_tensors_of_a_cache_are_written_into_not_replaced(name):
    """The calls go by the addresses of the tensors given at construction: an
    assignment of another tensor is refused, one in place is not."""
    cache = cpu_cache()
    t = getattr(cache, name)
    with pytest.raises(AttributeError, match="in place"):
        setattr(cache, name, t + 1)
    assert getattr(cache, name) is t
    with pytest.raises(AttributeError, match="in place"):
        setattr(cache, name, t.clone())
    if name == "lens":
        cache.lens += 2  # assigns the same tensor
    else:
        setattr(cache, name, t)
    assert getattr(cache, name) is t
    assert cache.lens.tolist() == ([2, 2, 2] if name == "lens" else [0, 0, 0])


def test_no_entries_need_no_addresses():
    """An empty tensor's address is null; with no entries nothing is done."""
    L, p = C.lib(), fake_pages()
    r = ct.byref(p)
    assert L.cg_pages_copy(r, r, None, None, 0, 0, None) == C.CG_OK
    assert L.cg_pages_fork(r, None, None, None, 0, 4096, 1 << 30, 0, None) == C.CG_OK
    assert L.cg_pages_free(r, None, 0, 0, None) == C.CG_OK
    # what else is wrong is still refused
    assert L.cg_pages_copy(r, None, None, None, 0, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_free(ct.byref(fake_pages(L=0)), None, 0, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_fork(r, None, None, None, 0, None, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_fork(r, None, None, None, 0, 4096, 16, 0, None) == C.CG_ERR_RANGE


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("nq", [1, 3])
def test_a_step_with_nothing_to_do(nq):
    """No request ended, none came, none is left: no error and no change."""
    cache, slots = make([40, 300], bt=16, Hkv=2)
    m = Model(cache)
    none = _ints([])
    cache.fork(none, none, none)
    cache.fork(none, none)
    cache.free(none)
    cache.copy(none, none)
    q = torch.empty((0, nq, 8, 128), dtype=torch.float16, device="cuda")
    lse = torch.empty((0, nq, 8), device="cuda")
    assert cache.attend(1, q, slots=none, lse=lse).shape == q.shape
    assert cache.attend(1, q, shared_slot=0, shared_blocks=1, out=q) is q
    with pytest.raises(ValueError):
        cache.attend(-1, q)
    with pytest.raises(ValueError):
        cache.attend(1, q, slots=slots)
    m.check(cache)


def test_a_growing_batch_holds_a_few_times_its_workspace(monkeypatch):
    """Workspaces that a captured graph may still use are kept; a batch that
    grows by a request at a time leaves few of them, four times the need in all."""
    cache, fake = host_cache(monkeypatch)
    sizes = []
    for R in range(1, 300):
        fake.ws_bytes = 1000 + 5000 * R
        cache.attend(0, torch.zeros((R, 1, 4, 64), dtype=torch.float16), slots=torch.zeros(R, dtype=torch.int32))
        name, args = fake.launched[-1]
        assert args[3] >= fake.ws_bytes
        sizes.append(args[3])
        held = cache._ws.numel() + sum(t.numel() for t in cache._outgrown)
        assert held <= 4 * fake.ws_bytes
    assert len(set(sizes)) <= 10 and sizes == sorted(sizes)


def test_the_sizes_kept_by_shape_do_not_grow_with_the_shared_blocks(monkeypatch):
    cache, fake = host_cache(monkeypatch)
    q = torch.zeros((2, 1, 4, 64), dtype=torch.float16)
    for shared in range(5):
        cache.attend(0, q, shared_blocks=shared)
    assert len(cache._attn) == 2  # with and without


def test_workspace_bytes_depend_on_whether_blocks_are_shared_alone():
    L, n = C.lib(), ct.c_size_t()
    for R, nq in ((1, 1), (4, 3), (60, 2)):
        sizes = set()
        for shared in (1, 2, 7, 12):
            a = fake_attention(n_requests=R, n_queries=nq, shared_blocks=shared)
            assert L.cg_attend_ws_bytes(ct.byref(fake_pages()), ct.byref(a), ct.byref(n)) == C.CG_OK
            sizes.add(n.value)
        assert len(sizes) == 1


def test_a_row_count_past_64_bits_is_refused():
    """2^31 queries of 2^31 heads for four requests are 2^64 rows: none, where
    the product wraps."""
    L, p, n = C.lib(), fake_pages(), ct.c_size_t()
    for nq, hq, R in ((1 << 31, 1 << 31, 4), (1 << 31, 1 << 31, 5), (1 << 31, 1 << 30, 1 << 3), (0xFFFFFFFF, 1, 1)):
        a = fake_attention(n_queries=nq, n_q_heads=hq, n_requests=R)
        assert L.cg_attend_ws_bytes(ct.byref(p), ct.byref(a), ct.byref(n)) == C.CG_ERR_INVALID_ARG, (nq, hq, R)


def test_numbers_that_the_kernels_cannot_count_to_are_refused():
    """The kernels step through slots and lists with 32-bit numbers: past 2^31
    a step could wrap and the loop not end."""
    L, n = C.lib(), ct.c_size_t()
    assert L.cg_pages_ws_bytes(ct.byref(fake_pages(n_slots=1 << 31)), ct.byref(n)) == C.CG_OK
    big = fake_pages(n_slots=(1 << 31) + 1)
    assert L.cg_pages_ws_bytes(ct.byref(big), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_fork(ct.byref(big), 4096, 4096, None, 0, 4096, 1 << 40, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_free(ct.byref(big), 4096, 0, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_compact(ct.byref(big), 4096, 4096, 16, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_free(ct.byref(fake_pages()), 4096, (1 << 31) + 1, 0, None) == C.CG_ERR_INVALID_ARG
