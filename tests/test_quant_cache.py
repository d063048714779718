"""The calls on a pool of 4 or 8 bits against the formulas in 64 bits.

Codes, scales and low values are compared bit for bit, and so are the values
read back.  Attention's tolerances are derived per element from the inputs (w
the softmax weights, u = half a step of the output's type, n tokens, and 2^-11
half a step of fp16; K_t = low + scale * code, |K|_t = |low| + scale * code):
  * a score is a sum of D products in fp32, in some order with at most two
    units of truncation a step, the sums of q with the low values in parts of
    22 bits: off by at most scale * (D * 2^-22 + 2^-20) * sum_d |q_d| |K|_td.
    A channel of q below 2^-25 of the largest may be lost, 2^-24 * max |q| *
    sum_d scale * code.  With es the sum of both over the worst token, a weight
    is off by a factor of at most 1 + 2 es;
  * where the shared blocks go through 16-bit values, K is rounded to 2^-11 of
    itself (fp16) or 2^-17 (bf16, in two parts), V and the weights to u;
  * a weight times a scale is rounded to fp16 once (2^-11), and below that
    type's normal range by at most 2^-29 of the largest weight times the
    group's largest scale: the codes' part is off by that times the code;
  * sums of n terms and the joins of pieces in fp32: n * 2^-23;
  * the result is rounded once: u |out|.
"""
import ctypes as ct
import math

import numpy as np
import pytest
import torch

from kv_cache_compression_decode_gb300 import codec as C
from kv_cache_compression_decode_gb300 import paged, synth
from tests.test_paged_pages import fake_pages

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
gpu = lambda f: pytest.mark.gpu(needs_gpu(f))  # noqa: E731
FP16, BF16 = torch.float16, torch.bfloat16
WORKSPACE_ROWS = 65  # query rows from which the shared blocks go through the workspace


def _ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# The format, plainly
# ---------------------------------------------------------------------------

def to_bits(x, dtype):
    """float64 numbers that the type holds exactly -> their 16 bits."""
    if dtype == FP16:
        return x.astype(np.float16).view(np.uint16)
    return (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def of_bits(b, dtype):
    if dtype == FP16:
        return b.view(np.float16).astype(np.float64)
    return (b.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x, dtype, bits, group):
    """x: float64 [..., C], finite numbers of the type -> codes [..., C], scale and low [..., C / group], by the
    definition: the scale is looked for among the type's numbers, a code among the integers."""
    top = 2 ** bits - 1
    y = x.reshape(x.shape[:-1] + (-1, group))
    low = y.min(-1, keepdims=True)
    d = (y.max(-1, keepdims=True) - low).astype(np.float32).astype(np.float64)
    grid = of_bits(np.arange(0x7C00 if dtype == FP16 else 0x7F80, dtype=np.uint16), dtype)  # ascending
    scale = grid[np.searchsorted(grid * top, d)]
    t = (y - low).astype(np.float32).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        n = np.floor(np.where(scale > 0, t / scale, 0.0))
    half = (n + 0.5) * scale  # exact
    n = np.where(t > half, n + 1, np.where((t == half) & (scale > 0) & (n % 2 == 1), n + 1, n))
    return n.reshape(x.shape).astype(np.uint8), scale[..., 0], low[..., 0]


def pack(codes, scale, low, dtype, bits, row):
    if bits == 4:
        codes = codes[..., 0::2] | codes[..., 1::2] << 4
    out = np.zeros(codes.shape[:-1] + (row,), np.uint16)
    n = codes.shape[-1] // 2
    out[..., :n] = np.ascontiguousarray(codes).view(np.uint16)
    out[..., n: n + 2 * scale.shape[-1]: 2] = to_bits(scale, dtype)
    out[..., n + 1: n + 2 * scale.shape[-1]: 2] = to_bits(low, dtype)
    return out


def parts(rows, cache):
    """int16 rows [..., row] on the GPU -> code, scale and low of every channel, float64 [..., C]."""
    f = cache._format
    Cc, n = f.n_kv_heads * f.head_dim, f.n_kv_heads * f.head_dim * f.bits // 16
    code = rows[..., :n].contiguous().view(torch.uint8)
    if f.bits == 4:
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    pairs = rows[..., n: n + 2 * (Cc // f.group)].contiguous().view(cache._type).double()
    return code.double(), pairs[..., 0::2].repeat_interleave(f.group, -1), pairs[..., 1::2].repeat_interleave(f.group, -1)


def test_the_plain_quantiser_by_hand():
    x = np.array([[0.0, 1.0, 2.0, 15.0] + [3.0] * 28])
    codes, scale, low = quantise(x, FP16, 4, 32)
    assert scale[0, 0] == 1 and low[0, 0] == 0 and codes[0, :5].tolist() == [0, 1, 2, 15, 3]
    x[0, 3] = 30.0  # scale 2: 1 and 3 lie on borders and go to the even code
    assert quantise(x, FP16, 4, 32)[0][0, :5].tolist() == [0, 0, 1, 15, 2]
    x[0, 3] = 15.01  # the next fp16 above 15.01 / 15
    codes, scale, low = quantise(x.astype(np.float16).astype(np.float64), FP16, 4, 32)
    assert scale[0, 0] == 1 + 2 ** -10
    codes, scale, low = quantise(np.full((1, 64), -2.5), BF16, 8, 64)
    assert scale[0, 0] == 0 and low[0, 0] == -2.5 and not codes.any()
    row = pack(*quantise(x, FP16, 4, 32), FP16, 4, 16)
    assert row[0, 0] == 0 | 1 << 4 | 2 << 8 | 15 << 12 and row[0, 8] == 0x3C01 and row[0, 9:].tolist() == [0] * 7


# ---------------------------------------------------------------------------
# Writing and reading
# ---------------------------------------------------------------------------

def empty(lens, bt, Hkv, D, bits, group, dtype, L=2, layout="plain", seed=0, slots=None):
    """A cache with blocks for sequences of `lens` tokens in slots 1 .. (or `slots`), the pool full of noise."""
    row = paged.QuantCache.row_width(Hkv, D, bits, group, dtype)
    need = [-(-n // bt) for n in lens]
    n_pool, n_slots = sum(need) + 5, len(lens) + 3
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = dict(plain=(L, n_pool, 2, bt, row), block_major=(n_pool, L, 2, bt, row), padded=(L, n_pool, 2, bt, row + 24))[layout]
    pool = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16)
    pool = pool.transpose(0, 1) if layout == "block_major" else pool[..., :row]
    ids = np.random.default_rng(seed).permutation(n_pool).tolist()
    order = slots if slots is not None else list(range(1, len(lens) + 1))
    table, all_lens, at = np.full((n_slots, max(need + [0]) + 2), -1, np.int32), np.zeros(n_slots, np.int32), 0
    for s, n, k in zip(order, lens, need):
        table[s, :k], all_lens[s] = ids[at: at + k], n
        at += k
    return paged.QuantCache(pool, _ints(table.reshape(-1)).view(table.shape), _ints(all_lens),
                            torch.ones(n_pool, dtype=torch.int32, device="cuda"), n_kv_heads=Hkv, head_dim=D, bits=bits,
                            group=group, dtype=dtype), _ints(order)


def rows_like(shape, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn(shape[-1], generator=g, device="cuda"))
    return (x + torch.randn(shape[-1], generator=g, device="cuda")).to(dtype)


def places(cache, slots, counts, start=None):
    """(row of k and v, block, row of the block) of every token."""
    tables, lens, bt = cache.tables.cpu().numpy(), cache.lens.cpu().numpy(), cache.block_tokens
    out, j = [], 0
    for i, (s, n) in enumerate(zip(slots.tolist(), counts)):
        first = lens[s] - n if start is None else start[i]
        out += [(j + k, tables[s, (first + k) // bt], (first + k) % bt) for k in range(n)]
        j += n
    return np.array(out, np.int64).reshape(-1, 3)


def want_rows(x, cache):
    f = cache._format
    return pack(*quantise(x.double().cpu().numpy(), cache._type, f.bits, f.group), cache._type, f.bits, cache.pool.shape[4])


FORMATS = [(4, 128, 128), (4, 128, 64), (4, 128, 32), (8, 128, 128), (8, 128, 64), (8, 128, 32), (4, 64, 64), (4, 64, 32),
           (8, 64, 64), (8, 64, 32)]


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("Hkv,bt,layout", [(1, 8, "plain"), (3, 16, "padded"), (8, 64, "block_major")])
def test_ragged_rows_are_stored_and_read_back(dtype, bits, D, group, Hkv, bt, layout):
    """Codes, scales and low values bit for bit; everything else of the pool and the rows of nobody as they were."""
    counts = [1, 0, 17, 5, 33]
    cache, slots = empty([1, 40, 20, 5, 64], bt, Hkv, D, bits, group, dtype, layout=layout)
    n, Cc = sum(counts), Hkv * D
    offsets = _ints(np.cumsum([2] + counts))  # two rows before the first sequence, four behind the last one
    k, v = rows_like((2, n + 6, Cc), dtype, 1), rows_like((2, n + 6, Cc), dtype, 2)
    before = cache.pool.clone()
    cache.write(k, v, slots=slots, offsets=offsets)
    at = torch.tensor(places(cache, slots, counts), device="cuda")
    pad = cache.pool.shape[4] - (Cc * bits // 16 + 2 * (Cc // group))
    for kv, x in enumerate((k, v)):
        got, want = cache.pool[:, at[:, 1], kv, at[:, 2]], want_rows(x[:, at[:, 0] + 2], cache)
        end = got.shape[-1] - pad
        assert np.array_equal(got.cpu().numpy().view(np.uint16)[..., :end], want[..., :end]), kv
        before[:, at[:, 1], kv, at[:, 2], :end] = got[..., :end]
    assert torch.equal(before, cache.pool)
    back = [torch.full((2, n + 6, Cc), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    cache.read(slots=slots, offsets=offsets, out=tuple(back))
    for kv, y in enumerate(back):
        code, scale, low = parts(cache.pool[:, at[:, 1], kv, at[:, 2]], cache)
        want = (code * scale + low).float().to(dtype)
        assert torch.equal(y[:, 2: 2 + n], want) and (y[:, :2] == 7).all() and (y[:, 2 + n:] == 7).all()
        x = (k, v)[kv][:, 2: 2 + n].double()
        assert ((code * scale + low - x).abs() <= scale / 2 * (1 + 2 ** -20) + x.abs() * 2 ** -23).all()
    cache.check()


@gpu
@pytest.mark.parametrize("R,n", [(1, 1), (5, 1), (3, 7)])
def test_an_even_share_a_start_and_strided_inputs(R, n):
    """Without offsets; k and v as slices of one projection's output; tokens from a given position on."""
    cache, slots = empty([50 + 3 * r for r in range(R)], 16, 2, 64, 4, 32, FP16, slots=list(range(R + 1, 1, -1)))
    both = rows_like((1, R * n, 5 * 128), FP16)
    k, v = both[..., 128:256], both[..., 384:512]
    start = [4 * r + 1 for r in range(R)]
    for kw in (dict(), dict(start=_ints(start))):
        cache.write(k, v, layer=1, slots=slots, **kw)
        at = torch.tensor(places(cache, slots, [n] * R, start if kw else None), device="cuda")
        for kv, x in enumerate((k, v)):
            got = cache.pool[1, at[:, 1], kv, at[:, 2]].cpu().numpy().view(np.uint16)
            assert np.array_equal(got, want_rows(x[0], cache))  # (128 channels in groups of 32: no padding)
        kb, vb = cache.read(layer=1, rows=R * n, slots=slots, **kw)
        code, scale, low = parts(cache.pool[1, at[:, 1], 0, at[:, 2]], cache)
        assert torch.equal(kb[0], (code * scale + low).half()) and vb.shape == k.shape
    cache.check()


@gpu
@pytest.mark.parametrize("bt", [1, 4])
@pytest.mark.parametrize("Hkv,D,group", [(1, 64, 32), (5, 64, 64), (40, 128, 128)])
def test_small_blocks_and_long_rows(bt, Hkv, D, group):
    """Rows of 8 to 640 eight-channel units, in blocks smaller than attention takes."""
    cache, slots = empty([3, 11], bt, Hkv, D, 8, group, FP16, L=3)
    k, v = rows_like((3, 10, Hkv * D), FP16), rows_like((3, 10, Hkv * D), FP16, 1)
    cache.write(k, v, slots=slots, offsets=_ints([0, 2, 10]))
    at = torch.tensor(places(cache, slots, [2, 8]), device="cuda")
    n = Hkv * D // 2 + 2 * (Hkv * D // group)
    for kv, x in enumerate((k, v)):
        got = cache.pool[:, at[:, 1], kv, at[:, 2]].cpu().numpy().view(np.uint16)
        assert np.array_equal(got[..., :n], want_rows(x, cache)[..., :n])
    back, _ = cache.read(n_layers=3, rows=10, slots=slots, offsets=_ints([0, 2, 10]))
    code, scale, low = parts(cache.pool[:, at[:, 1], 0, at[:, 2]], cache)
    assert torch.equal(back, (code * scale + low).float().half())
    cache.check()


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_on_borders_and_at_the_ends_of_the_type(dtype, bits):
    """Exact multiples of half a scale, constants, zeros of both signs, subnormals, one far value, the whole range."""
    rng = np.random.default_rng(0)
    top, most = 2 ** bits - 1, float(torch.finfo(dtype).max)
    least = float(torch.finfo(dtype).smallest_normal) * 2.0 ** (-10 if dtype == FP16 else -7)
    x = [np.concatenate([[0, top], rng.integers(0, 2 * top + 1, 30) / 2]) for _ in range(8)]      # scale 1
    x += [np.concatenate([[0, top * 0.75], rng.integers(0, 2 * top + 1, 30) * 0.375]) for _ in range(8)]
    x += [rng.integers(-9, 10, 32) * least, np.full(32, -1.5), np.zeros(32), -np.zeros(32), np.eye(1, 32, 3)[0] * 1000]
    x += [rng.integers(0, 2, 32) * least, np.where(rng.random(32) < 0.5, -most, most) * (1 if dtype == FP16 else 0.49),
          1.0 + rng.integers(0, 4, 32) * float(torch.finfo(dtype).eps), most - rng.integers(0, 3, 32) * most * 2.0 ** -6]
    x += [rng.standard_normal(32) * 2.0 ** e for e in range(-20, 12)]
    if len(x) % 4:
        x += [np.zeros(32)] * (4 - len(x) % 4)
    x = torch.tensor(np.stack(x).reshape(-1, 128), device="cuda").to(dtype)
    cache, slots = empty([x.shape[0]], 32, 1, 128, bits, 32, dtype)
    cache.write(x[None], x.flip(0)[None], slots=slots)
    at = torch.tensor(places(cache, slots, [x.shape[0]]), device="cuda")
    got = cache.pool[0, at[:, 1], 0, at[:, 2]]
    assert np.array_equal(got.cpu().numpy().view(np.uint16) & 0xFFFF, want_rows(x, cache) ) or same_but_zero_signs(got, x, cache)
    back, _ = cache.read(rows=x.shape[0], slots=slots)
    code, scale, low = parts(got, cache)
    want = (code * scale + low).float()
    want = torch.where(want.abs() > most, want.sign() * most, want).to(dtype)
    assert torch.equal(back[0], want) and torch.isfinite(back).all()
    cache.check()


def same_but_zero_signs(got, x, cache):
    """A group's low value may be either zero where it holds both."""
    code, scale, low = parts(got, cache)
    want = torch.tensor(want_rows(x, cache).view(np.int16), device="cuda")
    return all(torch.equal(a, b) for a, b in zip((code, scale, low), parts(want, cache)))


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits", [4, 8])
def test_a_group_that_is_not_finite_becomes_nan_and_is_flagged(dtype, bits):
    cache, slots = empty([6], 16, 2, 128, bits, 64, dtype)
    x = rows_like((1, 6, 256), dtype)
    x[0, 1, 70], x[0, 2, 0], x[0, 4, 255] = float("nan"), float("inf"), float("-inf")
    if dtype == BF16:
        x[0, 5, 130], x[0, 5, 131] = 3e38, -3e38  # their difference is not finite
    cache.write(x, x, slots=slots)
    k, v = cache.read(rows=6, slots=slots)
    bad = {(1, 1), (2, 0), (4, 3)} | ({(5, 2)} if dtype == BF16 else set())
    for y in (k, v):
        nan = torch.isnan(y[0].view(6, 4, 64))
        assert all(nan[i, g].all() if (i, g) in bad else not nan[i, g].any() for i in range(6) for g in range(4))
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_NONFINITE


@gpu
def test_rows_that_cannot_be_placed_are_flagged_and_left_out():
    """Slots and blocks out of range, more rows than tokens, tokens past the end; an empty sequence is no fault."""
    def fresh():
        return empty([20, 0, 20], 16, 1, 64, 4, 64, FP16, L=1)

    def run(cache, counts, flagged, used, **kw):
        n = sum(counts)
        x, before = rows_like((1, n, 64), FP16), cache.pool.clone()
        kw.setdefault("offsets", _ints(np.cumsum([0] + counts)))
        cache.write(x, x, **kw)
        changed = (before != cache.pool).any(-1).sum().item()
        out = tuple(torch.full((1, n, 64), 9.0, dtype=FP16, device="cuda") for _ in range(2))
        cache.read(out=out, **kw)
        assert (out[0] != 9).any(-1).sum().item() == used and changed == 2 * used
        if flagged:
            with pytest.raises(C.CodecError) as e:
                cache.check()
            assert e.value.code == C.CG_ERR_RANGE
        else:
            cache.check()

    run(fresh()[0], [3, 3, 3], False, 6, slots=_ints([1, 2, 3]))          # slot 2 is empty
    run(fresh()[0], [3, 3, 3], True, 6, slots=_ints([1, 6, 3]))           # there are six slots
    run(fresh()[0], [3, 3, 3], True, 6, slots=_ints([1, -1, 3]))
    run(fresh()[0], [21, 20, 1], True, 21, slots=_ints([1, 3, 1]))
    run(fresh()[0], [3, 4], True, 3, slots=_ints([1, 3]), start=_ints([17, 17]))
    run(fresh()[0], [3, 4], True, 3, slots=_ints([1, 3]), start=_ints([17, -2]))
    cache, _ = fresh()
    cache.tables[1, 1] = 1000
    run(cache, [20], True, 16, slots=_ints([1]))
    cache, _ = fresh()
    cache.lens[1] = 1 << 30
    run(cache, [2], True, 0, slots=_ints([1]))
    run(fresh()[0], [4, 2], False, 2, slots=_ints([1, 3]), offsets=_ints([4, 4, 6]))  # the first four are nobody's
    run(fresh()[0], [4, 2], False, 2, slots=_ints([1, 3]), offsets=_ints([0, 0, 2]))  # the last four


@gpu
def test_many_sequences_and_a_long_context():
    """More sequences than a block keeps; four units a thread over several layers; a stream of its own; twice alike."""
    counts = [r % 3 for r in range(1500)]
    cache, slots = empty([n + 1 for n in counts], 8, 1, 64, 4, 64, FP16, L=1)
    x = rows_like((1, sum(counts), 64), FP16)
    cache.write(x, x, slots=slots, offsets=_ints(np.cumsum([0] + counts)))
    at = torch.tensor(places(cache, slots, counts), device="cuda")
    got = cache.pool[0, at[:, 1], 1, at[:, 2]].cpu().numpy().view(np.uint16)
    assert np.array_equal(got[:, :18], want_rows(x[0], cache)[:, :18])

    cache, slots = empty([2011], 64, 8, 128, 8, 128, BF16, L=6)
    k, v = rows_like((5, 2011, 1024), BF16), rows_like((5, 2011, 1024), BF16, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cache.write(k, v, layer=1, slots=slots, stream=s)
    once = cache.read(layer=1, n_layers=5, rows=2011, slots=slots, stream=s)
    s.synchronize()
    at = torch.tensor(places(cache, slots, [2011]), device="cuda")
    for l in (0, 4):
        got = cache.pool[1 + l, at[:, 1], 0, at[:, 2]].cpu().numpy().view(np.uint16)
        assert np.array_equal(got[:, :528], want_rows(k[l], cache)[:, :528])
        code, scale, low = parts(cache.pool[1 + l, at[:, 1], 1, at[:, 2]], cache)
        assert torch.equal(once[1][l], (code * scale + low).float().to(BF16))
    pool = cache.pool.clone()
    cache.write(k, v, layer=1, slots=slots)
    assert torch.equal(pool, cache.pool)
    cache.check()


@gpu
def test_nothing_to_write_or_read():
    cache, slots = empty([20], 16, 1, 64, 4, 64, FP16)
    pool = cache.pool.clone()
    x = torch.empty((1, 0, 64), dtype=FP16, device="cuda")
    cache.write(x, x, slots=slots)
    cache.write(rows_like((1, 4, 64), FP16), rows_like((1, 4, 64), FP16), slots=_ints([]), offsets=_ints([0]))
    k, v = cache.read(rows=3, slots=_ints([]), offsets=_ints([0]))
    assert k.shape == (1, 3, 64) and not k.any() and not v.any() and torch.equal(pool, cache.pool)
    cache.check()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def make(lens, shared_blocks=0, bt=16, Hkv=2, D=128, bits=4, group=None, dtype=FP16, layout="plain", L=2, seed=0, spare=9):
    """A cache whose slot 0 is the shared context and whose further slots are the requests (lens: tokens of each,
    shared ones included).  Rows of the pool that belong to no token hold noise."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    P, n_slots, Cc = shared_blocks * bt, len(lens) + 3, Hkv * D
    row = paged.QuantCache.row_width(Hkv, D, bits, group, dtype)
    need = [max(0, -(-(n - P) // bt)) if n else 0 for n in lens]
    n_pool = shared_blocks + sum(need) + spare
    ids = np.random.default_rng(seed).permutation(n_pool).tolist()
    table = np.full((n_slots, shared_blocks + max(need + [0]) + 2), -1, np.int32)
    table[0, :shared_blocks] = ids[:shared_blocks]
    at = shared_blocks
    shape = dict(plain=(L, n_pool, 2, bt, row), block_major=(n_pool, L, 2, bt, row), padded=(L, n_pool, 2, bt, row + 24))[layout]
    pool = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda", dtype=torch.int16)
    pool = pool.transpose(0, 1) if layout == "block_major" else pool[..., :row]
    all_lens = np.zeros(n_slots, np.int32)
    all_lens[0] = P
    for s, (n, k) in enumerate(zip(lens, need), 1):
        table[s, :shared_blocks] = ids[:shared_blocks]
        table[s, shared_blocks: shared_blocks + k] = ids[at: at + k]
        at += k
        all_lens[s] = n
    cache = paged.QuantCache(pool, _ints(table.reshape(-1)).view(table.shape), _ints(all_lens),
                             torch.ones(n_pool, dtype=torch.int32, device="cuda"), n_kv_heads=Hkv, head_dim=D, bits=bits,
                             group=group, dtype=dtype)
    sigma = torch.exp(0.5 * torch.randn(Cc, generator=g, device="cuda"))
    mean = 0.5 * torch.randn(Cc, generator=g, device="cuda") * sigma
    for s, n in [(0, P)] + [(s, n) for s, n in enumerate(lens, 1)]:
        first = 0 if s == 0 else P
        if n > first:
            k, v = (torch.randn((L, n - first, Cc), generator=g, device="cuda") * sigma + mean for _ in range(2))
            cache.write(k.to(dtype), v.to(dtype), slots=_ints([s]))
    return cache, _ints(range(1, len(lens) + 1))


def check(cache, q, out, lse, slots, layer, scale, shared_blocks=0):
    tables, lens = cache.tables.cpu().numpy(), cache.lens.cpu().numpy()
    R, nq, Hq, D = q.shape
    f, bt = cache._format, cache.block_tokens
    Hkv, g, u = f.n_kv_heads, Hq // f.n_kv_heads, torch.finfo(q.dtype).eps / 2
    through = shared_blocks > 0 and R * nq * g >= WORKSPACE_ROWS
    code, sc, low = (x.view(x.shape[:-1] + (Hkv, D)) for x in parts(cache.pool[layer], cache))
    qd = q.double()
    for r, s in enumerate(slots.tolist()):
        n = int(lens[s])
        blocks = _ints(tables[s][: -(-n // bt)]).long()
        rows = [x[blocks].permute(1, 0, 2, 3, 4).reshape(2, -1, Hkv, D)[:, :n] for x in (code, sc, low)]
        for i in range(nq):
            seen = n - nq + 1 + i
            if seen <= 0:
                assert (out[r, i] == 0).all() and (lse[r, i] == -math.inf).all(), (r, i)
                continue
            (kc, vc), (ks, vs), (kl, vl) = ([x[j, :seen] for j in range(2)] for x in rows)
            h = lambda x: x.view(Hkv, g, D)  # noqa: E731
            qq = h(qd[r, i])
            x = torch.einsum("hgd,thd->hgt", qq, kl + ks * kc) * scale
            worst = (torch.einsum("hgd,thd->hgt", qq.abs(), kl.abs() + ks * kc).amax(2) * (D * 2.0 ** -22 + 2.0 ** -20)
                     + 2.0 ** -24 * qq.abs().amax(2) * (ks * kc).sum(2).amax(0)[:, None])
            if through:
                worst = worst + (2.0 ** -11 if q.dtype == FP16 else 2.0 ** -17) * torch.einsum(
                    "hgd,thd->hgt", qq.abs(), (kl + ks * kc).abs()).amax(2)
            es = abs(scale) * worst
            w = torch.softmax(x, 2)
            V = vl + vs * vc
            ref, A = torch.einsum("hgt,thd->hgd", w, V), torch.einsum("hgt,thd->hgd", w, vl.abs() + vs * vc)
            B = torch.einsum("hgt,thd->hgd", w, vs * vc)
            full = rows[1][1].amax(0)  # the largest scales of the sequence, those unseen included
            tiny = seen * 2.0 ** -29 * w.amax(2)[..., None] * (full * (2 ** f.bits - 1))[:, None]
            if through:
                A = A + torch.einsum("hgt,thd->hgd", w, V.abs()) * 2 * u / 2.0 ** -20
                tiny = tiny + seen * 2.0 ** -25 * w.amax(2)[..., None] * V.abs().amax(0)[:, None]
            tol = u * ref.abs() + 2.0 ** -11 * B + (2 * es[..., None] + seen * 2.0 ** -23 + 2.0 ** -20) * A + tiny + 2.0 ** -25
            err = (h(out[r, i].double()) - ref).abs()
            assert (err <= tol).all(), (r, i, float((err / tol).max()))
            want = torch.logsumexp(x, 2)
            tol = es + (seen + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -22
            err = (lse[r, i].double().view(Hkv, g) - want).abs()
            assert (err <= tol).all(), (r, i, float((err / tol).max()))


def attend(cache, slots, nq=1, Hq=8, layer=1, scale=None, shared_blocks=0, seed=3, q=None, out=None, **kw):
    R = slots.shape[0]
    if q is None:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        q = (1.5 * torch.randn((R, nq, Hq, cache._hd), generator=g, device="cuda")).to(cache._type)
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    if out is None:
        out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    cache.attend(layer, q, slots=slots, shared_slot=0, shared_blocks=shared_blocks, scale=scale, out=out, lse=lse, **kw)
    return q, out, lse


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 300, 1000]


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits,D,group", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,nq,bt", [(8, 8, 1, 16), (14, 2, 3, 8), (40, 1, 5, 64), (3, 3, 2, 256), (8, 1, 1, 32)])
def test_own_tokens_only(dtype, bits, D, group, Hq, Hkv, nq, bt):
    cache, slots = make(LENS, bt=bt, Hkv=Hkv, D=D, bits=bits, group=group, dtype=dtype)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("bits,D,group", [(4, 128, 128), (4, 128, 32), (8, 64, 64)])
@pytest.mark.parametrize("Hq,Hkv,nq", [(16, 2, 1), (2, 2, 1), (14, 2, 3), (40, 1, 5)])
@pytest.mark.parametrize("bt,shared", [(8, 1), (16, 70), (64, 5), (256, 3)])
def test_shared_blocks(dtype, bits, D, group, Hq, Hkv, nq, bt, shared):
    P = shared * bt
    lens = [P + max(n, nq - 1) if n or nq == 1 else 0 for n in LENS if n != 1] + [0, P + nq]
    cache, slots = make(lens, shared, bt, Hkv, D, bits, group, dtype, seed=shared)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5, shared)


@gpu
@pytest.mark.parametrize("R", [1, 5, 33, 130])
@pytest.mark.parametrize("nq,Hq,D,dtype", [(1, 8, 128, FP16), (4, 16, 128, BF16), (1, 16, 64, BF16)])
def test_batches_over_a_long_context(R, nq, Hq, D, dtype):
    """From a few query rows on the shared blocks to many tiles of them; with one, several and very unequal lengths."""
    P, bt = 1500 // 32 * 32, 32
    lens = [P + nq + (37 * r) % 200 for r in range(R)]
    lens[R // 2] = P + 2500
    cache, slots = make(lens, P // bt, bt, 1, D, dtype=dtype, seed=R)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq, shared_blocks=P // bt)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5, P // bt)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("R,g,bits,group", [(8, 8, 4, 128), (16, 8, 4, 32), (30, 4, 8, 64), (40, 8, 4, 64)])
def test_query_rows_around_one_tile_over_thousands_of_shared_tokens(dtype, R, g, bits, group):
    """64 to 320 rows of two KV heads on 6000 tokens: k_quant_rows, and through the workspace in one and in two tiles."""
    lens = [6016 + 1 + 3 * r for r in range(R)]
    cache, slots = make(lens, 6016 // 32, 32, 2, 128, bits, group, dtype, seed=R)
    q, out, lse = attend(cache, slots, Hq=2 * g, shared_blocks=6016 // 32)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5, 6016 // 32)


@gpu
@pytest.mark.parametrize("Hkv,D,pieces", [(8, 64, n) for n in (1, 2, 8, 9, 12, 31, 32, 33, 36, 37, 64, 65, 151, 160)]
                         + [(1, 64, n) for n in (1, 2, 5, 40)] + [(4, 128, n) for n in (17, 129)])
def test_one_request_in_few_and_many_pieces(Hkv, D, pieces):
    """The pieces that the join of one request's rows meets: fewer and more than its warps take in one and in several goes
    (of eight heads a piece a block, of four two, of one eight)."""
    tokens = max(1, 32 * (2 * pieces - 3) - 5)  # two places of 32 tokens a block, three of them for the beginning
    cache, slots = make([tokens], bt=32, Hkv=Hkv, D=D, bits=4, group=64, seed=pieces)
    q, out, lse = attend(cache, slots, Hq=2 * Hkv)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5)


@gpu
@pytest.mark.parametrize("Hkv,g,nq", [(4, 8, 1), (8, 8, 4), (12, 1, 1), (5, 5, 2), (6, 5, 2), (32, 1, 1), (9, 3, 7)])
@pytest.mark.parametrize("D,shared", [(128, 0), (128, 9), (64, 0), (64, 9)])
def test_groups_of_heads(Hkv, g, nq, D, shared):
    lens = [9 * 16 + n for n in (nq, 40, 333, 700)]
    cache, slots = make(lens, shared, 16, Hkv, D, group=32)
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hkv * g, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, D ** -0.5, shared)


@gpu
@pytest.mark.parametrize("shared", [0, 6])
def test_a_prompt_over_its_context(shared):
    """Hundreds of query tokens, each seeing one more."""
    cache, slots = make([700, 500], shared, 16, 2, 128)
    q, out, lse = attend(cache, slots, nq=333, Hq=4, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5, shared)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("shared,Hkv,nq", [(0, 4, 4), (6, 4, 4), (6, 1, 9), (0, 2, 2)])
def test_a_token_reaches_only_the_queries_that_see_it(dtype, shared, Hkv, nq):
    """The last token's scales and low values become infinite, NaN or huge: only the last query may tell."""
    n = 6 * 16 + 40
    cache, slots = make([n], shared, 16, Hkv, 128, group=64, dtype=dtype)
    q, out, lse = attend(cache, slots, nq=nq, Hq=4 * Hkv, shared_blocks=shared)
    block = int(cache.tables[1, (n - 1) // 16])
    at = Hkv * 128 // 4
    big = to_bits(np.array([1e4 if dtype == FP16 else 1e30]), dtype).view(np.int16)[0]
    inf, nan = (0x7C00, 0x7E00) if dtype == FP16 else (0x7F80, 0x7FC0)
    for value in (inf, nan, int(big)):
        for kv in range(2):
            for word in range(2):
                was = cache.pool[1, block, kv, (n - 1) % 16].clone()
                cache.pool[1, block, kv, (n - 1) % 16, at + word] = value
                _, o, e = attend(cache, slots, nq=nq, q=q, shared_blocks=shared)
                cache.pool[1, block, kv, (n - 1) % 16] = was
                if value != int(big):
                    assert torch.equal(o[:, :-1], out[:, :-1]) and torch.equal(e[:, :-1], lse[:, :-1]), (value, kv, word)
                    assert not torch.isfinite(o[0, -1, :4, :64]).all() or (kv == 0 and torch.isfinite(e[0, -1, :4]).all()), (value, kv, word)
                else:  # the same weights in other units: operands below fp16's normal range may round otherwise
                    u = torch.finfo(dtype).eps
                    assert torch.allclose(o[:, :-1].float(), out[:, :-1].float(), rtol=u, atol=u * float(out.float().abs().max()))
                    assert torch.allclose(e[:, :-1], lse[:, :-1], rtol=2.0 ** -20)
                assert torch.equal(o[:, -1, 4:], out[:, -1, 4:])  # the other heads
    cache.check()


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_scales_of_very_different_size(dtype):
    """Groups and tokens whose values lie many octaves apart, in both orders along the sequence."""
    n, e = 200, 9 if dtype == FP16 else 30
    cache, slots = make([n, n], 0, 16, 1, 128, group=32, dtype=dtype)
    t = torch.arange(n, device="cuda")
    x = rows_like((2, 2 * n, 128), dtype).float()
    by = torch.exp2(torch.cat([t * e / n - e / 2, e / 2 - t * e / n]).round())[:, None]
    by = by * torch.exp2(torch.tensor([0, -5, 3, -2], device="cuda").repeat_interleave(32))
    k = rows_like((2, 2 * n, 128), dtype, 5)
    cache.write(k, (x * by).to(dtype), slots=slots)
    q, out, lse = attend(cache, slots, Hq=8)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("dtype,size", [(FP16, 2.0 ** -18), (FP16, 3e4), (BF16, 1e-20), (BF16, 1e20)])
def test_queries_of_any_size(dtype, size):
    cache, slots = make([100, 300], 0, 16, 2, 128, dtype=dtype)
    q = rows_like((2, 1, 8, 128), dtype).float()
    q = (q / q.abs().max() * size).to(dtype)
    scale = 128 ** -0.5 / size if dtype == BF16 or size > 1 else 100.0
    q, out, lse = attend(cache, slots, q=q, scale=scale)
    cache.check()
    check(cache, q, out, lse, slots, 1, np.float32(scale).item())


@gpu
@pytest.mark.parametrize("R", [3, 40])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (0.0, 1e-30), (1e-20, 1.0), (3.0, 1.0), (-3.0, 1.0), (1e-30, 1e-30)])
def test_scales(R, scale, size):
    lens = [5 * 16 + 1 + 37 * r % 90 for r in range(R)]
    cache, slots = make(lens, 5, 16, 2, 64, dtype=BF16)
    q = (rows_like((R, 2, 8, 64), BF16).float() * size).to(BF16)
    q, out, lse = attend(cache, slots, nq=2, q=q, scale=scale, shared_blocks=5)
    cache.check()
    check(cache, q, out, lse, slots, 1, np.float32(scale).item(), 5)


@gpu
@pytest.mark.parametrize("dtype", [FP16, BF16])
def test_scores_that_rise_over_values_without_size(dtype):
    """V is zero, or a constant, for most tokens while the scores climb by hundreds of octaves; then they fall again."""
    n = 640
    cache, slots = make([n, n], 0, 16, 1, 128, group=32, dtype=dtype)
    t = torch.arange(n, device="cuda")
    ramp = torch.cat([t, n - t]).float()[:, None] * 0.5
    k = ramp.expand(-1, 128) + rows_like((2 * n, 128), dtype, 4).float() * 0.01
    v = torch.zeros((2 * n, 128), device="cuda")
    v[:, 32:64] = -2.5
    v[::7] = rows_like((2 * n, 128), dtype, 5).float()[::7]
    cache.write(*(x.to(dtype).expand(2, -1, -1) for x in (k, v)), slots=slots)
    q = torch.ones((2, 1, 8, 128), dtype=dtype, device="cuda") * torch.tensor([1, 2, -1, 0, 0.25, 8, -8, 0.01], device="cuda").to(dtype)[:, None]
    q, out, lse = attend(cache, slots, q=q, scale=0.125)
    cache.check()
    assert torch.isfinite(out).all()
    check(cache, q, out, lse, slots, 1, 0.125)


@gpu
def test_a_query_that_is_not_finite_spoils_its_own_row_alone():
    cache, slots = make([300], 0, 16, 2, 64)
    q, out, lse = attend(cache, slots, nq=2)
    bad = q.clone()
    bad[0, 1, 3, 7] = float("nan")
    bad[0, 0, 6, 0] = float("inf")
    _, o, e = attend(cache, slots, nq=2, q=bad)
    keep = torch.ones((2, 8), dtype=torch.bool, device="cuda")
    keep[1, 3] = keep[0, 6] = False
    assert torch.equal(o[0][keep], out[0][keep]) and torch.equal(e[0][keep], lse[0][keep])
    assert torch.isnan(o[0, 1, 3]).all() and not torch.isfinite(o[0, 0, 6]).all()
    cache.check()


@gpu
@pytest.mark.parametrize("layout", ["block_major", "padded"])
@pytest.mark.parametrize("shared,R", [(0, 9), (9, 9), (9, 70)])
def test_layouts_strides_and_slot_order(layout, shared, R):
    lens = [9 * 16 + 3 + 11 * r for r in range(R)]
    cache, slots = make(lens, shared, 16, 4, 64, layout=layout)
    slots = slots.flip(0).contiguous()
    both = torch.randn((R, 2, 8, 2, 64), device="cuda").half()
    q = both[:, :, :, 1]
    out = torch.zeros((2, R, 8, 64), dtype=FP16, device="cuda").transpose(0, 1)
    q, out, lse = attend(cache, slots, q=q, out=out, shared_blocks=shared, scale=-0.2)
    cache.check()
    check(cache, q, out, lse, slots, 1, np.float32(-0.2).item(), shared)


@gpu
def test_default_slots_and_no_lse():
    cache, _ = make([40, 100], 0, 16, 2, 64)
    cache.lens[0] = 0
    q = torch.randn((3, 1, 4, 64), device="cuda").half()
    out = cache.attend(1, q)
    lse = torch.empty((3, 1, 4), device="cuda")
    assert torch.equal(cache.attend(1, q, lse=lse), out)
    check(cache, q, out, lse, _ints([0, 1, 2]), 1, 0.125)
    assert cache.attend(1, q[:0]).shape == (0, 1, 4, 64)
    cache.check()


@gpu
@pytest.mark.parametrize("shared", [0, 6])
def test_same_bits_every_time(shared):
    lens = [6 * 16 + n for n in (5, 800, 33, 1500, 90)]
    cache, slots = make(lens, shared, 16, 2, 128, group=32)
    q, out, lse = attend(cache, slots, shared_blocks=shared)
    for _ in range(3):
        _, o, e = attend(cache, slots, q=q, shared_blocks=shared)
        assert torch.equal(o, out) and torch.equal(e, lse)
    cache.check()


@gpu
@pytest.mark.parametrize("R", [4, 70])
def test_graph_replays_with_new_tokens_and_another_stream(R):
    """A captured decode step (write one token, attend) is replayed as the sequences grow."""
    shared, bt = 5, 16
    lens = [shared * bt + 1 + r % 7 for r in range(R)]
    cache, slots = make([n + 30 for n in lens], shared, bt, 2, 64, group=32)
    cache.lens[1: R + 1] = _ints(lens)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    k, v, q = (torch.zeros(s, dtype=FP16, device="cuda") for s in ((1, R, 128), (1, R, 128), (R, 1, 8, 64)))
    out, lse = torch.empty_like(q), torch.empty((R, 1, 8), device="cuda")
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
    for _ in range(3):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        cache.lens[slots.long()] += 1
        graph.replay()
        torch.cuda.synchronize()
        check(cache, q, out, lse, slots, 1, 0.125, shared)
    cache.check()


@gpu
@pytest.mark.parametrize("R", [2, 70])
def test_refused_requests_and_blocks_outside_the_pool(R):
    cache, slots = make([5 * 16 + 20] * R, 5, 16, 2, 64)
    cache.lens[1] = 5 * 16 - 1  # does not see the shared blocks
    q, out, lse = attend(cache, slots, shared_blocks=5)
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_RANGE and (out[0] == 0).all() and (lse[0] == -math.inf).all()
    check(cache, q[1:], out[1:], lse[1:], slots[1:], 1, 0.125, 5)
    cache.lens[1] = 5 * 16 + 20
    for bad in (4000, -1, 2 ** 31 - 1):
        for row, col in ((0, 2), (2, 5)):
            was = int(cache.tables[row, col])
            cache.tables[row, col] = bad
            attend(cache, slots, q=q, shared_blocks=5)
            with pytest.raises(C.CodecError) as e:
                cache.check()
            assert e.value.code == C.CG_ERR_RANGE
            cache.tables[row, col] = was
    _, out, lse = attend(cache, slots, q=q, shared_blocks=5)
    cache.check()
    check(cache, q, out, lse, slots, 1, 0.125, 5)


@gpu
@pytest.mark.parametrize("R", [2, 70])
def test_offsets_past_32_bits(R):
    """Blocks whose words lie past 2^32 of a layer, written, read and attended to."""
    bt, Hkv, D = 256, 32, 128
    row = paged.QuantCache.row_width(Hkv, D)
    n_pool = (1 << 32) // (2 * bt * row) + 20
    pool = torch.empty((1, n_pool, 2, bt, row), dtype=torch.int16, device="cuda")
    table = torch.full((R + 1, 3), -1, dtype=torch.int32)
    table[:, 0] = n_pool - 1
    if R == 2:
        table[1:, 1] = torch.arange(R) + n_pool - 4
    else:
        table[1:, 1] = n_pool - 2
    shared = 1
    cache = paged.QuantCache(pool, table.cuda(), _ints([bt] + [bt + 40] * R), torch.ones(n_pool, dtype=torch.int32, device="cuda"),
                             n_kv_heads=Hkv, head_dim=D)
    k, v = rows_like((1, bt, Hkv * D), FP16), rows_like((1, bt, Hkv * D), FP16, 1)
    cache.write(k, v, slots=_ints([0]))
    for r in range(1, R + 1 if R == 2 else 2):
        cache.write(k[:, r: r + 40], v[:, r: r + 40], slots=_ints([r]))
    back, _ = cache.read(rows=40, slots=_ints([1]))
    code, scale, low = parts(cache.pool[0, int(table[1, 1]), 0, :40], cache)
    assert torch.equal(back[0], (code * scale + low).half())
    assert ((code * scale + low - k[0, 1:41]).abs() <= scale / 2).all()  # the format's bound
    q, out, lse = attend(cache, _ints(range(1, R + 1)), Hq=Hkv, layer=0, shared_blocks=shared)
    cache.check()
    kv = cache.pool[:, int(table[0, 0]) - 8:].clone()  # the blocks in use, as a small pool
    small = paged.QuantCache(kv, (cache.tables - (int(table[0, 0]) - 8)).clamp(min=-1), cache.lens, cache.refs[-kv.shape[1]:].contiguous(),
                             n_kv_heads=Hkv, head_dim=D)
    small.tables[cache.tables < 0] = -1
    check(small, q, out, lse, _ints(range(1, R + 1)), 0, D ** -0.5, shared)


# ---------------------------------------------------------------------------
# Together: a decoded context, forked, continued, freed, compacted
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_a_decoded_context_is_forked_and_continued(bits, group):
    L, T, Hkv, D, bt, R = 3, 333, 2, 64, 16, 5
    cfg = C.Config(L, T, Hkv * D)
    kv = synth.ar1_kv(L, T, Hkv * D, 0.95, 2, 0, device="cuda")
    enc = C.encode(cfg, kv)
    dec = C.decode(cfg, enc)
    cache = paged.QuantCache.empty(L, 60, bt, Hkv, D, R + 1, 30, bits, group)
    cache.fork(_ints([-1]), _ints([0]), _ints([T]))
    cache.decode(cfg, enc, 0)
    k, v = cache.read(n_layers=L, rows=T, slots=_ints([0]))
    at = torch.tensor(places(cache, _ints([0]), [T]), device="cuda")
    for kvi, y in enumerate((k, v)):
        code, scale, low = parts(cache.pool[:, at[:, 1], kvi, at[:, 2]], cache)
        assert torch.equal(y, (code * scale + low).half())
        assert ((y - dec[:, kvi]).abs().double() <= scale / 2 + y.abs().double() * 2 ** -10 + 2 ** -24).all()
    slots = _ints(range(1, R + 1))
    cache.fork(_ints([0] * R), slots, _ints([40] * R))
    for step in range(3):
        cache.lens[1:] += step + 1
        n = (step + 1) * R
        new = [rows_like((L, n, Hkv * D), FP16, 10 * step + i) for i in range(2)]
        cache.write(*new, slots=slots)
        q, out, lse = attend(cache, slots, nq=step + 1, layer=2, shared_blocks=T // bt, seed=step)
        check(cache, q, out, lse, slots, 2, D ** -0.5, T // bt)
    cache.free(slots[::2].contiguous())
    cache.compact()
    left = slots[1::2].contiguous()
    q = q[1::2].contiguous()
    check(cache, *attend(cache, left, nq=3, q=q, layer=2, shared_blocks=T // bt), left, 2, D ** -0.5, T // bt)
    cache.check()
    other = paged.QuantCache.empty(L, 10, bt, Hkv, D, 1, 5, bits, group)
    other.copy(_ints([int(cache.tables[2, 0])]), _ints([3]), source=cache)
    assert torch.equal(other.pool[:, 3], cache.pool[:, int(cache.tables[2, 0])])
    with pytest.raises(ValueError):
        other.copy(_ints([0]), _ints([0]), source=paged.QuantCache.empty(L, 10, bt, Hkv, D, 1, 5, bits, group, dtype=BF16))


@gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_the_example_on_a_quantised_pool(bits):
    """After 2 x 5 steps, a free and a compaction, the last step's outputs are the formula's over the codes as they are."""
    from examples import shared_prefix

    cache, slots, q, out = shared_prefix.run(layers=2, context=333, kv_heads=2, q_heads=8, head_dim=64, block_tokens=16,
                                             requests=6, steps=5, bits=bits, log=lambda s: None)
    assert [cache.lens.tolist()[s] for s in slots.tolist()] == [343] * 3 and cache._format.bits == bits
    for layer in range(2):
        _, again, lse = attend(cache, slots, q=q[layer], layer=layer, shared_blocks=333 // 16)
        assert torch.equal(again, out[layer])
        check(cache, q[layer], out[layer], lse, slots, layer, 0.125, 333 // 16)


# ---------------------------------------------------------------------------
# Refusals on the host
# ---------------------------------------------------------------------------

def fake_format(**kw):
    d = dict(dtype=0, bits=4, group=64, n_kv_heads=1, head_dim=64)
    d.update(kw)
    return C.cg_quant(*[d[f] for f, _ in C.cg_quant._fields_])


def quant_pages(**kw):
    """Made-up addresses; 64 channels in 4 bits are rows of 24 words."""
    d = dict(C=24, token_stride=24, kv_stride=16 * 24, block_stride=2 * 16 * 24, layer_stride=40 * 2 * 16 * 24)
    d.update(kw)
    return fake_pages(**d)


def fake_rows(**kw):
    d = dict(k=1 << 30, v=1 << 31, slots=1 << 20, first=None, start=None, n_seqs=2, n_rows=4, layer=0, n_layers=2)
    d.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    r = C.cg_token_rows(*[d[f] for f, _ in C.cg_token_rows._fields_[:9]])
    r.k_stride, r.v_stride = (ct.c_uint64 * 2)(*kw.get("k_stride", (256, 64))), (ct.c_uint64 * 2)(*kw.get("v_stride", (256, 64)))
    return r


def fake_attention(**kw):
    d = dict(q=1 << 30, out=1 << 31, lse=None, slots=None, dtype=0, n_requests=2, n_queries=1, n_q_heads=4, n_kv_heads=1, head_dim=64,
             layer=0, shared_slot=0, shared_blocks=0, scale=1.0)
    d.update(kw)
    a = C.cg_attention()
    for k, v in d.items():
        setattr(a, k, v)
    a.q_stride = a.out_stride = (ct.c_uint64 * 3)(256, 256, 64)
    return a


@pytest.mark.parametrize("f,words", [(dict(), 24), (dict(bits=8), 40), (dict(group=32), 24), (dict(n_kv_heads=8, head_dim=128, group=128), 272),
                                     (dict(n_kv_heads=8, head_dim=128, group=32), 320), (dict(n_kv_heads=3, group=32, bits=8), 112)])
def test_width_of_a_row(f, words):
    n = ct.c_uint32()
    assert C.lib().cg_quant_row(ct.byref(fake_format(**f)), ct.byref(n)) == C.CG_OK and n.value == words
    assert C.lib().cg_quant_row(ct.byref(fake_format(**f)), None) == C.CG_ERR_INVALID_ARG


BAD_FORMAT = [dict(dtype=2), dict(bits=2), dict(bits=16), dict(group=16), dict(group=128), dict(group=48), dict(n_kv_heads=0), dict(head_dim=32),
              dict(head_dim=256), dict(n_kv_heads=1 << 21)]


@pytest.mark.parametrize("kw", BAD_FORMAT)
def test_bad_formats_are_refused_on_the_host(kw):
    L, p, f, n, w = C.lib(), quant_pages(), fake_format(**kw), ct.c_uint32(), ct.c_size_t()
    assert L.cg_quant_row(ct.byref(f), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_write(ct.byref(p), ct.byref(f), ct.byref(fake_rows()), 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_read(ct.byref(p), ct.byref(f), ct.byref(fake_rows()), 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend_ws_bytes(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), ct.byref(w)) == C.CG_ERR_INVALID_ARG


@pytest.mark.parametrize("pool", [dict(C=32, token_stride=32), dict(pool=None), dict(pool=(1 << 30) + 8), dict(tables=None), dict(lens=None),
                                  dict(lens=(1 << 21) + 2), dict(token_stride=20), dict(token_stride=28), dict(block_stride=772), dict(kv_stride=388),
                                  dict(layer_stride=4), dict(block_tokens=12), dict(n_blocks=1 << 28), dict(L=0), dict(n_pool_blocks=0)])
def test_bad_pools_are_refused_on_the_host(pool):
    L, p, f, r, w = C.lib(), quant_pages(**pool), fake_format(), fake_rows(n_layers=1), ct.c_size_t()
    for call in (L.cg_quant_write, L.cg_quant_read):
        assert call(ct.byref(p), ct.byref(f), ct.byref(r), 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend_ws_bytes(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), ct.byref(w)) == C.CG_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=(1 << 30) + 8), dict(v=(1 << 31) + 2), dict(n_rows=5), dict(layer=2), dict(n_layers=0),
                                dict(n_layers=3), dict(layer=1, n_layers=0xFFFFFFFF), dict(slots=(1 << 20) + 1), dict(first=(1 << 20) + 2),
                                dict(start=(1 << 20) + 2), dict(k_stride=(256, 63)), dict(v_stride=(252, 64)), dict(n_rows=(1 << 31) + 2),
                                dict(n_seqs=0xFFFFFFFF)])
def test_bad_rows_are_refused_on_the_host(kw):
    L, p, f, r = C.lib(), quant_pages(), fake_format(), fake_rows(**kw)
    for call in (L.cg_quant_write, L.cg_quant_read):
        assert call(ct.byref(p), ct.byref(f), ct.byref(r), 0, None) == C.CG_ERR_INVALID_ARG
    # nothing to do is no error, and enqueues nothing
    for kw in (dict(n_seqs=0), dict(n_rows=0), dict(n_rows=0, k=None)):
        assert L.cg_quant_write(ct.byref(p), ct.byref(f), ct.byref(fake_rows(**kw)), 0, None) == C.CG_OK


@pytest.mark.parametrize("kw", [dict(dtype=1), dict(n_kv_heads=2), dict(head_dim=128), dict(n_q_heads=0), dict(q=None), dict(out=(1 << 31) + 8), dict(layer=2),
                                dict(shared_blocks=13), dict(shared_blocks=1, shared_slot=8), dict(scale=float("nan")), dict(n_requests=0)])
def test_bad_attention_is_refused_on_the_host(kw):
    L, p, f, n = C.lib(), quant_pages(), fake_format(), ct.c_size_t()
    assert L.cg_quant_attend_ws_bytes(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), ct.byref(n)) == C.CG_OK
    assert L.cg_quant_attend(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), 4096, n.value - 1, 0, None) == C.CG_ERR_RANGE
    assert L.cg_quant_attend(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), 4096 + 128, n.value, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend(ct.byref(p), ct.byref(f), ct.byref(fake_attention()), None, n.value, 0, None) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend_ws_bytes(ct.byref(p), ct.byref(f), ct.byref(fake_attention(**kw)), ct.byref(n)) == C.CG_ERR_INVALID_ARG
    assert L.cg_quant_attend(ct.byref(p), ct.byref(f), ct.byref(fake_attention(**kw)), 4096, 1 << 30, 0, None) == C.CG_ERR_INVALID_ARG


def test_python_checks():
    i32 = dict(dtype=torch.int32)
    state = torch.zeros((3, 4), **i32), torch.zeros(3, **i32), torch.zeros(5, **i32)
    pool = torch.zeros((2, 5, 2, 16, 24), dtype=torch.int16)
    form = dict(n_kv_heads=1, head_dim=64)
    for p, kw in ((pool.half(), form), (pool[..., :16], form), (pool, dict(form, bits=8)), (pool, dict(form, dtype=torch.float32)), (pool[0], form)):
        with pytest.raises(ValueError):
            paged.QuantCache(p, *state, torch.zeros(1, **i32), **kw)
    for kw in (dict(form, bits=5), dict(form, group=128), dict(form, head_dim=96)):
        with pytest.raises(C.CodecError):
            paged.QuantCache(pool, *state, torch.zeros(1, **i32), **kw)
    cache = paged.QuantCache(pool, *state, torch.zeros(1, **i32), **form)
    assert cache.channels == 64 and cache.block_tokens == 16
    x, ids = torch.zeros((1, 4, 64), dtype=FP16), lambda *v: torch.tensor(v, **i32)
    for args, kw in (((x.bfloat16(), x), {}), ((x[0], x[0]), {}), ((x[..., :32], x[..., :32]), {}), ((x, x[:, :2]), {}), ((x, x), dict(layer=-1)),
                     ((x, x), dict(slots=ids(0, 1), offsets=ids(0, 4))), ((x, x), dict(slots=ids(0), start=ids(0, 1))),
                     ((x, x), dict(offsets=ids())), ((x, x), dict(offsets=ids(0, 1, 2, 3, 4))), ((x, x), dict(slots=ids(0).long())),
                     ((x.transpose(1, 2).contiguous().transpose(1, 2), x), {})):
        with pytest.raises(ValueError):
            cache.write(*args, **kw)
    with pytest.raises(ValueError, match="rows or out"):
        cache.read()
    with pytest.raises(ValueError, match="are those of out"):
        cache.read(out=(x, x), rows=3)
    with pytest.raises(ValueError, match="not in GPU memory"):
        cache.write(x, x, slots=ids(0))
    with pytest.raises(ValueError):
        cache.attend(0, torch.zeros((1, 1, 4, 64), dtype=BF16))


def test_packed_arguments_are_laid_out_as_the_structures():
    want = [C.cg_token_rows(1, 2, 3, 4, 5, 6, 7, 8, 9, (ct.c_uint64 * 2)(10, 11), (ct.c_uint64 * 2)(12, 13)),
            C.cg_attention(*range(1, 14), (ct.c_uint64 * 3)(14, 15, 16), (ct.c_uint64 * 3)(17, 18, 19), 0.5)]
    got = [paged._pack_rows(*range(1, 14)), paged._pack_attention(*range(1, 20), 0.5)]
    for a, b in zip(want, got):
        assert bytes(a) == b
