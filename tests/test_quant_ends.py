"""Caches in 4 or 8 bits at the ends of the types' ranges.  Tolerances are those of test_quant_cache.py."""
import numpy as np
import pytest
import torch

import tests.test_paged_attend as plain
from kv_cache_compression_decode_gb300 import codec as C
from tests.test_quant_cache import BF16, attend, check, empty, gpu, make, parts, places, rows_like


@gpu
@pytest.mark.parametrize("group", [32, 128])
def test_the_top_code_past_the_largest_number_reads_back_as_that(group):
    """bf16, 4 bits: the largest code's value may lie past 2^128 although every channel is finite."""
    most, unit = float(torch.finfo(BF16).max), 2.0 ** 120
    rng = np.random.default_rng(1)
    x = rng.uniform(-4, 255, (64, 128)) * unit
    low = np.linspace(-3, 4, 64)
    x[:, 0::32], x[:, 1::32] = low[:, None] * unit, most
    x[:, 2::32] = np.maximum(x[:, 2::32], low[:, None] * unit)
    x = torch.tensor(np.maximum(x, low[:, None] * unit), device="cuda").to(BF16)
    cache, slots = empty([64], 32, 1, 128, 4, group, BF16)
    cache.write(x[None], -x[None], slots=slots)
    at = torch.tensor(places(cache, slots, [64]), device="cuda")
    y = x.double().view(64, -1, group)
    odd = torch.isinf((y.amax(-1) - y.amin(-1)).float()).repeat_interleave(group, 1)  # such a span is stored as NaN, and flagged
    assert odd.any()
    for kv, y in enumerate(cache.read(rows=64, slots=slots)):
        code, scale, first = parts(cache.pool[0, at[:, 1], kv, at[:, 2]], cache)
        value = code * scale + first
        assert torch.equal(torch.isnan(value), odd)
        if kv == 0:
            assert (value >= 2.0 ** 128).any()
        assert torch.equal(torch.isnan(y[0]), odd) and torch.equal(y[0][~odd], value.clamp(max=most).float().to(BF16)[~odd])
    with pytest.raises(C.CodecError) as e:
        cache.check()
    assert e.value.code == C.CG_ERR_NONFINITE


@gpu
@pytest.mark.parametrize("R", [8, 80])
def test_keys_past_the_largest_number_reach_the_queries_that_use_them(R):
    """bf16: groups whose top code lies past 2^128, and queries that are zero in their channels."""
    shared, bt, Hkv = 160, 32, 8
    cache, slots = make([shared * bt + 1 + r % 5 for r in range(R)], shared, bt, Hkv, 128, group=32, dtype=BF16)
    k, v = rows_like((1, shared * bt, Hkv * 128), BF16, 1), rows_like((1, shared * bt, Hkv * 128), BF16, 2)
    q = rows_like((R, 1, Hkv, 128), BF16, 3)
    k.view(-1, Hkv, 128)[::7, :, 0:32] = 2.0 ** 120
    k.view(-1, Hkv, 128)[::7, :, 3] = torch.finfo(BF16).max
    q[..., 0:32] = 0.0
    cache.write(k, v, layer=1, slots=slots.new_zeros(1))
    q, out, lse = attend(cache, slots, q=q, shared_blocks=shared)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5, shared)


@gpu
@pytest.mark.parametrize("R", [2, 40])
@pytest.mark.parametrize("bits", [16, 4])
def test_scales_below_1e_35(bits, R):
    """Products of 2^116 at a scale of 2^-118, which makes ordinary scores of them, and at a scale of zero."""
    P, Hkv, D, size = 96, 2, 64, 2.0 ** 57
    lens = [P + 2 + 7 * r % 50 for r in range(R)]
    q = (rows_like((R, 2, 8, D), BF16, 7).double() * 2.0 ** 56).to(BF16)
    if bits == 16:
        cache, slots = plain.make(lens, P // 16, 16, Hkv, D, BF16)
        cache.pool.mul_(size)
    else:
        cache, slots = make(lens, P // 16, 16, Hkv, D, dtype=BF16)
        for s, n in [(0, P)] + [(s, n - P) for s, n in enumerate(lens, 1)]:
            rows = [(rows_like((2, n, Hkv * D), BF16, 2 * s + i).double() * size).to(BF16) for i in range(2)]
            cache.write(*rows, slots=torch.tensor([s], dtype=torch.int32, device="cuda"))
    for scale in (2.0 ** -118, 0.0, -2.0 ** -118):
        if bits == 16:
            _, out, lse = plain.attend(cache, slots, nq=2, Hq=8, D=D, q=q, scale=scale, shared_blocks=P // 16)
            cache.check()
            plain.check(cache, q, out, lse, slots, 1, scale)
        else:
            _, out, lse = attend(cache, slots, nq=2, q=q, scale=scale, shared_blocks=P // 16)
            cache.check()
            check(cache, q, out, lse, slots, 1, scale, P // 16)


@gpu
@pytest.mark.parametrize("nq,Hq", [(1, 8), (3, 16)])
@pytest.mark.parametrize("e", [-132, -126, -110, -100, 96, 111, 113, 116, 118, 126])
def test_queries_over_the_whole_range_of_bf16(e, nq, Hq):
    """Channels up to 2^e in size, and a scale that makes ordinary scores of them."""
    cache, slots = make([100, 300], 0, 16, 2, 128, dtype=BF16)
    q = rows_like((2, nq, Hq, 128), BF16).double()
    q = (q / q.abs().max() * 1.9 * 2.0 ** e).to(BF16)
    scale = float(np.float32(min(128 ** -0.5 * 2.0 ** -e, 2.0 ** 125)))
    q, out, lse = attend(cache, slots, nq=nq, q=q, scale=scale)
    cache.check()
    check(cache, q, out, lse, slots, 1, scale)


@gpu
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("e", [-100, -80, 80, 105, 114, 118])
def test_keys_over_the_whole_range_of_bf16(e, group):
    """Keys of about 2^e against queries of about 2^-e."""
    cache, slots = make([100, 300], 0, 16, 2, 128, group=group, dtype=BF16)
    k, v = rows_like((2, 400, 256), BF16, 1), rows_like((2, 400, 256), BF16, 2)
    cache.write((k.double() * 2.0 ** e).to(BF16), v, slots=slots, offsets=torch.tensor([0, 100, 400], dtype=torch.int32, device="cuda"))
    q = (rows_like((2, 1, 8, 128), BF16, 3).double() * 2.0 ** -e).to(BF16)
    q, out, lse = attend(cache, slots, q=q)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("nq,Hq", [(1, 8), (3, 16)])
@pytest.mark.parametrize("bits,group", [(4, 128), (8, 32)])
def test_values_near_the_end_of_bf16(nq, Hq, bits, group):
    """Values of V up to 2^117: forty tokens of nearly the same weight."""
    cache, slots = make([40, 33], 0, 16, 2, 128, bits, group, BF16)
    v = torch.randn((2, 73, 256), generator=torch.Generator("cuda").manual_seed(4), device="cuda").clamp(-2, 2)
    k = torch.randn((2, 73, 256), generator=torch.Generator("cuda").manual_seed(5), device="cuda") * 0.1
    cache.write(k.to(BF16), (v.double() * 2.0 ** 116).to(BF16), slots=slots, offsets=torch.tensor([0, 40, 73], dtype=torch.int32, device="cuda"))
    q, out, lse = attend(cache, slots, nq=nq, Hq=Hq)
    cache.check()
    check(cache, q, out, lse, slots, 1, 128 ** -0.5)


@gpu
@pytest.mark.parametrize("nq", [1, 3])
def test_scores_that_rise_over_large_constant_values(nq):
    """bf16: groups whose channels are all 2^90 (scale 0) while the scores climb by hundreds of octaves."""
    n = 640
    cache, slots = make([n, n], 0, 16, 1, 128, group=32, dtype=BF16)
    t = torch.arange(n, device="cuda")
    k = torch.cat([t, n - t]).float()[:, None].expand(-1, 128) * 0.5
    v = torch.full((2 * n, 128), 2.0 ** 90, device="cuda")
    v[:, 32:64] = 1.5
    cache.write(*(x.to(BF16).expand(2, -1, -1) for x in (k, v)), slots=slots)
    by = torch.tensor([1, 2, -1, 0, 0.25, 0.125, -0.5, 0.01], device="cuda").to(BF16)
    q = by[:, None].expand(2, nq, 8, 128).contiguous()
    q, out, lse = attend(cache, slots, nq=nq, q=q, scale=0.03125)
    cache.check()
    check(cache, q, out, lse, slots, 1, 0.03125)


@gpu
@pytest.mark.parametrize("R", [2, 40])
@pytest.mark.parametrize("bits", [16, 4])
def test_queries_of_zero_at_the_largest_scale(bits, R):
    """A scale of 3e38 times log2 e lies past fp32: a score of zero is zero all the same, and the answer the mean."""
    P, Hkv, D, scale = 96, 2, 64, 3e38
    lens = [P + 1 + 7 * r % 50 for r in range(R)]
    q = torch.zeros((R, 1, 8, D), dtype=BF16, device="cuda")
    if bits == 16:
        cache, slots = plain.make(lens, P // 16, 16, Hkv, D, BF16)
        _, out, lse = plain.attend(cache, slots, Hq=8, D=D, q=q, scale=scale, shared_blocks=P // 16)
        cache.check()
        plain.check(cache, q, out, lse, slots, 1, scale)
    else:
        cache, slots = make(lens, P // 16, 16, Hkv, D, dtype=BF16)
        _, out, lse = attend(cache, slots, q=q, scale=scale, shared_blocks=P // 16)
        cache.check()
        check(cache, q, out, lse, slots, 1, scale, P // 16)
