"""Page calls on the sequences of a paged pool (cg_pages_copy / _fork / _free
/ _compact) against a plain model of the state in numpy, bit for bit."""
import ctypes as ct

import numpy as np
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged, synth

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
NB = -1


def _ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


class Model:
    """The state in numpy; pool is the 16-bit patterns [L][n_pool][2][bt][C]."""

    def __init__(self, cache):
        self.pool = cache.pool.cpu().view(torch.int16).numpy().copy()
        self.tables, self.lens, self.refs = (t.cpu().numpy().copy() for t in (cache.tables, cache.lens, cache.refs))
        self.bt = cache.block_tokens

    def fork(self, parent, child, reserve):
        free = [b for b in range(len(self.refs)) if self.refs[b] == 0]
        at = 0
        before = self.lens.copy()
        for p, c, rv in zip(parent, child, reserve):
            n = int(before[p]) if p >= 0 else 0
            full, total = n // self.bt, -(-(n + rv) // self.bt)
            fresh = free[at: at + total - full]
            at += total - full
            row = [int(b) for b in self.tables[p][:full]] if full else []
            if n % self.bt:
                self.pool[:, fresh[0], :, : n % self.bt] = self.pool[:, self.tables[p][full], :, : n % self.bt]
            for b in row:
                self.refs[b] += 1
            for b in fresh:
                self.refs[b] = 1
            self.tables[c] = row + fresh + [NB] * (self.tables.shape[1] - total)
            self.lens[c] = n

    def free(self, slots):
        for s in slots:
            for b in self.tables[s]:
                if b >= 0:
                    self.refs[b] -= 1
            self.tables[s] = NB
            self.lens[s] = 0

    def compact(self):
        live = np.flatnonzero(self.refs)
        src = [b for b in live if b >= len(live)]
        dst = [b for b in range(len(live)) if self.refs[b] == 0]
        remap = np.where(self.refs > 0, np.arange(len(self.refs)), NB).astype(np.int32)
        for s, d in zip(src, dst):
            self.pool[:, d] = self.pool[:, s]
            remap[s], self.refs[d], self.refs[s] = d, self.refs[s], 0
        self.tables = np.where(self.tables >= 0, remap[np.maximum(self.tables, 0)], self.tables)
        return remap

    def check(self, cache):
        cache.check()
        assert np.array_equal(cache.tables.cpu().numpy(), self.tables)
        assert np.array_equal(cache.lens.cpu().numpy(), self.lens)
        assert np.array_equal(cache.refs.cpu().numpy(), self.refs)
        assert np.array_equal(cache.pool.cpu().view(torch.int16).numpy(), self.pool)


def _fill(pool, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pool.view(torch.int16).random_(-30000, 30000, generator=g)  # any pattern, NaNs among them
    return pool


def _pool(layout, L, n_pool, bt, Cc, seed=0):
    """Pools whose addresses are multiples of 16, 8, 4 and 2 bytes, and block-major."""
    if layout == "plain":
        return _fill(torch.empty((L, n_pool, 2, bt, Cc), dtype=torch.float16, device="cuda"), seed)
    if layout == "block_major":
        return _fill(torch.empty((n_pool, L, 2, bt, Cc), dtype=torch.float16, device="cuda"), seed).transpose(0, 1)
    if layout == "kv_major":
        x = _fill(torch.empty((2, L, n_pool, bt, Cc), dtype=torch.float16, device="cuda"), seed)
        return x.permute(1, 2, 0, 3, 4)
    pad = int(layout[3:])  # token rows longer than C: "pad64", "pad4", "pad2", "pad1"
    return _fill(torch.empty((L, n_pool, 2, bt, Cc + pad), dtype=torch.float16, device="cuda"), seed)[..., :Cc]


def _cache(layout="plain", L=2, n_pool=40, bt=16, Cc=64, slots=8, width=12, seed=0):
    c = paged.PagedCache.empty(1, n_pool, bt, 1, slots, width)
    return paged.PagedCache(_pool(layout, L, n_pool, bt, Cc, seed), c.tables, c.lens, c.refs)


LAYOUTS = ["plain", "block_major", "kv_major", "pad64", "pad4", "pad2", "pad1"]


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("bt,Cc", [(16, 64), (1, 32), (64, 1024), (8, 33)])
def test_fork_free_compact_match_the_model(layout, bt, Cc):
    """A context, forks of it at lengths on and off a block border, forks of
    forks, ends and a compaction."""
    rng = np.random.default_rng(bt + Cc)
    for n in (0, 1, bt - 1, bt, bt + 1, 3 * bt + bt // 2):
        cache = _cache(layout, bt=bt, Cc=Cc, seed=n)
        held = set(rng.choice(40, 6, replace=False).tolist())  # blocks of somebody else: holes in the numbering
        cache.refs[torch.tensor(sorted(held), device="cuda")] = 1
        m = Model(cache)
        for parent, child, reserve in (([-1], [2], [n + bt]), ([2, 2, -1], [5, 0, 3], [1, 0, 2 * bt]),
                                       ([5, 0], [7, 1], [3, bt])):
            cache.fork(_ints(parent), _ints(child), _ints(reserve))
            m.fork(parent, child, reserve)
            if parent == [-1]:
                cache.lens[2] = n
                m.lens[2] = n
            m.check(cache)
        cache.free(_ints([2, 7]))
        m.free([2, 7])
        m.check(cache)
        remap = cache.compact()
        assert np.array_equal(remap.cpu().numpy(), m.compact())
        # the blocks of somebody else have moved with the rest
        m.check(cache)
        cache.free(_ints([0, 1, 3, 5, 4]))
        m.free([0, 1, 3, 5, 4])
        m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_fork_without_reserve_and_of_many():
    cache = _cache(n_pool=9000, slots=2500, width=4, L=1, Cc=8)
    m = Model(cache)
    cache.fork(_ints([-1]), _ints([0]), _ints([40]))
    m.fork([-1], [0], [40])
    cache.lens[0] = 40
    m.lens[0] = 40
    child = np.random.default_rng(0).permutation(np.arange(1, 2500)).tolist()
    cache.fork(_ints([0] * 2499), _ints(child))
    m.fork([0] * 2499, child, [0] * 2499)
    m.check(cache)
    cache.free(_ints(child[::2]))
    m.free(child[::2])
    m.check(cache)
    assert np.array_equal(cache.compact().cpu().numpy(), m.compact())
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_copy_matches_the_model(layout):
    cache = _cache(layout, L=3, n_pool=23, bt=8, Cc=40)
    m = Model(cache)
    src, dst = [3, 3, 22, 0], [1, 2, 7, 21]
    cache.copy(_ints(src), _ints(dst))
    m.pool[:, dst] = m.pool[:, src]
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_copy_between_pools_of_different_layouts():
    a, b = _cache("pad2", n_pool=9, seed=1), _cache("block_major", n_pool=30, seed=2)
    ma, mb = Model(a), Model(b)
    b.copy(_ints([8, 0, 4]), _ints([29, 0, 12]), source=a)
    mb.pool[:, [29, 0, 12]] = ma.pool[:, [8, 0, 4]]
    mb.check(b)
    ma.check(a)
    # ids are checked against their own pool: 20 is no block of `a`, 30 none of `b`
    b.copy(_ints([20, 1, 2]), _ints([3, 30, 5]), source=a)
    mb.pool[:, 5] = ma.pool[:, 2]
    with pytest.raises(C.CodecError) as e:
        b.check()
    assert e.value.code == C.CG_ERR_RANGE
    mb.check(b)


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("what,parent,child,reserve", [
    ("parent out of range", [0, 8], [1, 2], [1, 1]), ("child out of range", [0, 0], [1, 8], [1, 1]),
    ("child not empty", [0, 0], [1, 0], [1, 1]), ("child named twice", [0, 0], [1, 1], [1, 1]),
    ("row too short", [0, 0], [1, 2], [1, 12 * 16]), ("pool too small", [0] * 5, [1, 2, 3, 4, 5], [115] * 5),
    ("sum past 32 bits", [0] * 5, [1, 2, 3, 4, 5], [2 ** 31 - 1] * 5)])
def test_a_refused_fork_changes_nothing(what, parent, child, reserve):
    cache = _cache()
    cache.fork(_ints([-1]), _ints([0]), _ints([20]))
    cache.lens[0] = 20
    m = Model(cache)
    cache.fork(_ints(parent), _ints(child), _ints(reserve))
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE, what
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_fork_that_leaves_three_blocks():
    """Five children of 7 fresh blocks each out of 38: the refusal above is not early."""
    cache = _cache()
    cache.fork(_ints([-1]), _ints([0]), _ints([20]))
    cache.lens[0] = 20
    m = Model(cache)
    cache.fork(_ints([0] * 5), _ints([1, 2, 3, 4, 5]), _ints([100] * 5))
    m.fork([0] * 5, [1, 2, 3, 4, 5], [100] * 5)
    m.check(cache)
    assert int((cache.refs == 0).sum()) == 3


@pytest.mark.gpu
@needs_gpu
def test_free_of_empty_repeated_and_bad_slots():
    cache = _cache()
    cache.fork(_ints([-1, -1]), _ints([0, 3]), _ints([20, 33]))
    cache.lens[0], cache.lens[3] = 20, 33
    m = Model(cache)
    cache.free(_ints([3, 3, 6, 3]))
    m.free([3])
    m.check(cache)
    cache.free(_ints([8, 0]))
    m.free([0])
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_corrupt_tables_are_flagged_and_stay_in_bounds():
    cache = _cache()
    cache.fork(_ints([-1, -1]), _ints([0, 3]), _ints([40, 33]))
    cache.lens[0] = 40
    cache.tables[0, 1] = 4000  # a full block outside the pool
    m = Model(cache)
    cache.fork(_ints([0]), _ints([1]), _ints([0]))
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_CORRUPT
    assert cache.tables[1].tolist()[1] == NB and cache.lens[1].item() == 40
    assert np.array_equal(cache.refs.cpu().numpy()[m.tables[0][[0, 2]]], [2, 1])
    cache.free(_ints([0]))
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_CORRUPT
    cache.refs[cache.tables[3][0].long()] = 0  # a reference lost: its count does not wrap
    cache.free(_ints([3]))
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_CORRUPT
    assert int(cache.refs.min()) == 0 and int(cache.refs.max()) == 1
    cache.tables[5, 2] = 39  # names a free block
    cache.compact()
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_CORRUPT
    assert cache.tables[5, 2].item() == NB


@pytest.mark.gpu
@needs_gpu
def test_page_calls_on_another_stream_and_in_a_graph():
    cache = _cache(n_pool=60)
    cache.fork(_ints([-1]), _ints([0]), _ints([44]))
    cache.lens[0] = 44
    parent, child, reserve, ended = _ints([0, 0]), _ints([4, 6]), _ints([9, 30]), _ints([4])
    remap = torch.empty(60, dtype=torch.int32, device="cuda")
    m = Model(cache)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cache.fork(parent, child, reserve)
        cache.free(ended)
        cache.compact(remap)
    m.check(cache)  # nothing has run yet
    with torch.cuda.stream(s):
        graph.replay()
    torch.cuda.synchronize()
    m.fork([0, 0], [4, 6], [9, 30])
    m.free([4])
    want = m.compact()
    m.check(cache)
    assert np.array_equal(remap.cpu().numpy(), want)
    cache.free(_ints([6]), stream=s)
    s.synchronize()
    m.free([6])
    m.check(cache)


@pytest.mark.gpu
@needs_gpu
def test_offsets_past_32_bits():
    """Blocks whose element offsets lie past 2^32 in a pool."""
    bt, Cc, n_pool, gap = 16, 64, 7, 1 << 30
    flat = torch.empty(6 * gap + 2 * bt * Cc, dtype=torch.float16, device="cuda")
    pool = flat.as_strided((1, n_pool, 2, bt, Cc), (flat.numel(), gap, bt * Cc, Cc, 1))
    pool.copy_(torch.randn((1, n_pool, 2, bt, Cc), device="cuda"))
    c = paged.PagedCache.empty(1, n_pool, bt, 1, 3, 4)
    cache = paged.PagedCache(pool, c.tables, c.lens, c.refs)
    want = pool.clone()
    cache.copy(_ints([0, 6]), _ints([5, 1]))
    cache.refs[torch.tensor([5, 6], device="cuda")] = 1
    cache.tables[1, 0], cache.tables[1, 1] = 6, 5
    cache.compact()
    cache.check()
    want[:, 5], want[:, 1] = want[:, 0].clone(), want[:, 6].clone()
    want[:, 0], want[:, 1] = want[:, 5].clone(), want[:, 6].clone()
    assert torch.equal(pool, want)
    assert cache.tables[1].tolist()[:2] == [1, 0]


# ---------------------------------------------------------------------------
# Refusals on the host (no GPU)
# ---------------------------------------------------------------------------

def fake_pages(**kw):
    """Made-up, never dereferenced addresses."""
    d = dict(pool=1 << 30, L=2, C=64, n_pool_blocks=40, block_tokens=16, layer_stride=40 * 2 * 16 * 64,
             kv_stride=16 * 64, block_stride=2 * 16 * 64, token_stride=64, tables=1 << 20, lens=1 << 21, refs=1 << 22,
             n_slots=8, n_blocks=12)
    d.update(kw)
    return C.cg_pages(*[d[f] for f, _ in C.cg_pages._fields_])


BAD_STATE = [dict(pool=None), dict(pool=(1 << 30) + 1), dict(L=0), dict(C=0), dict(n_pool_blocks=0),
             dict(n_pool_blocks=0xFFFFFFFF), dict(block_tokens=0), dict(block_tokens=12), dict(token_stride=63),
             dict(tables=None), dict(lens=None), dict(refs=None), dict(tables=(1 << 20) + 2), dict(n_slots=0),
             dict(n_blocks=0), dict(n_blocks=1 << 28)]


@pytest.mark.parametrize("kw", BAD_STATE)
def test_bad_state_is_refused_on_the_host(kw):
    L, p, n = C.lib(), fake_pages(**kw), ct.c_size_t()
    assert L.cg_pages_ws_bytes(ct.byref(fake_pages()), ct.byref(n)) == C.CG_OK and n.value % 256 == 0
    assert L.cg_pages_ws_bytes(ct.byref(p), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_fork(ct.byref(p), 4096, 4096, None, 1, 4096, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_free(ct.byref(p), 4096, 1, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_pages_compact(ct.byref(p), 4096, 4096, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG


def test_bad_arguments_are_refused_on_the_host():
    L, p, n = C.lib(), fake_pages(), ct.c_size_t()
    bad, rng = C.CG_ERR_INVALID_ARG, C.CG_ERR_RANGE
    assert L.cg_pages_ws_bytes(ct.byref(p), ct.byref(n)) == C.CG_OK
    assert L.cg_pages_ws_bytes(ct.byref(p), None) == bad and L.cg_pages_ws_bytes(None, ct.byref(n)) == bad
    r, ws, big = ct.byref(p), 4096, 1 << 30
    assert L.cg_pages_fork(r, None, 4096, None, 1, ws, big, 0, None) == bad
    assert L.cg_pages_fork(r, 4096, 4098, None, 1, ws, big, 0, None) == bad
    assert L.cg_pages_fork(r, 4096, 4096, 4097, 1, ws, big, 0, None) == bad
    assert L.cg_pages_fork(r, 4096, 4096, None, 9, ws, big, 0, None) == bad  # more children than slots
    assert L.cg_pages_fork(r, 4096, 4096, None, 1, ws + 128, big, 0, None) == bad
    assert L.cg_pages_fork(r, 4096, 4096, None, 1, None, big, 0, None) == bad
    assert L.cg_pages_fork(r, 4096, 4096, None, 1, ws, n.value - 1, 0, None) == rng
    assert L.cg_pages_free(r, None, 1, 0, None) == bad and L.cg_pages_free(r, 4098, 1, 0, None) == bad
    assert L.cg_pages_compact(r, None, ws, big, 0, None) == bad
    assert L.cg_pages_compact(r, 4096, ws + 8, big, 0, None) == bad
    assert L.cg_pages_compact(r, 4096, ws, n.value - 1, 0, None) == rng
    assert L.cg_pages_copy(r, None, 4096, 4096, 1, 0, None) == bad
    assert L.cg_pages_copy(r, r, 4096, None, 1, 0, None) == bad
    for kw in (dict(L=3), dict(C=32), dict(block_tokens=32)):
        assert L.cg_pages_copy(r, ct.byref(fake_pages(**kw)), 4096, 4096, 1, 0, None) == bad
    # nothing to do is no error, and enqueues nothing
    assert L.cg_pages_copy(r, r, 4096, 4096, 0, 0, None) == C.CG_OK
    assert L.cg_pages_fork(r, 4096, 4096, None, 0, ws, big, 0, None) == C.CG_OK
    assert L.cg_pages_free(r, 4096, 0, 0, None) == C.CG_OK


def test_python_checks():
    i32 = dict(dtype=torch.int32)
    pool = torch.zeros((2, 5, 2, 16, 64), dtype=torch.float16)
    tables, lens, refs = torch.zeros((3, 4), **i32), torch.zeros(3, **i32), torch.zeros(5, **i32)
    for args in ((pool.float(), tables, lens, refs), (pool[0], tables, lens, refs),
                 (pool.transpose(3, 4), tables, lens, refs), (pool, tables.long(), lens, refs),
                 (pool, tables, lens[:2], refs), (pool, tables, lens, refs[:4]), (pool, tables[:, ::2], lens, refs)):
        with pytest.raises(ValueError):
            paged.PagedCache(*args)
    cache = paged.PagedCache(pool, tables, lens, refs)
    one, two = torch.zeros(1, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError):
        cache.fork(one, two)
    with pytest.raises(ValueError):
        cache.fork(one.long(), one.long())
    with pytest.raises(ValueError):
        cache.copy(one, two)
    with pytest.raises(ValueError):
        cache.compact(two)
    for call in (lambda: cache.fork(one, one), lambda: cache.free(one), lambda: cache.compact(), lambda: cache.copy(one, one)):
        with pytest.raises(ValueError, match="not in GPU memory"):  # every tensor here is a CPU tensor
            call()
    q = torch.zeros((2, 1, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="not in GPU memory"):
        cache.attend(0, q)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q, slots=one), dict(q=q, out=q[:1]), dict(q=q, lse=q),
               dict(q=q, shared_blocks=-1), dict(q=torch.zeros((4, 1, 4, 64), dtype=torch.float16))):
        with pytest.raises(ValueError):
            cache.attend(0, **kw)


@pytest.mark.gpu
@needs_gpu
def test_context_decodes_into_a_forked_slot():
    """fork gives a slot its blocks, decode fills them: reading the slot's
    rows back gives the linear decode bit for bit."""
    L, T, Cc, bt = 2, 333, 64, 16
    cfg = C.Config(L, T, Cc, 10, T, 128, C.layer_steps(L))
    enc = C.encode(cfg, synth.ar1_kv(L, T, Cc, 0.95, 1, seed=7).cuda())
    cache = _cache(n_pool=50, slots=3, width=30)
    cache.refs[::2] = 1
    cache.fork(_ints([-1]), _ints([1]), _ints([T]))
    cache.decode(cfg, enc, 1)
    cache.check()
    n = -(-T // bt)
    row = cache.tables[1].tolist()
    assert row[:n] == list(range(1, 2 * n, 2)) and set(row[n:]) == {NB} and cache.lens.tolist() == [0, T, 0]
    got = cache.pool[:, row[:n]].permute(0, 2, 1, 3, 4).reshape(L, 2, n * bt, Cc)[:, :, :T]
    assert torch.equal(got.view(torch.int16), C.decode(cfg, enc).view(torch.int16))
