"""One encoded context, continued by a batch of requests.

    python examples/shared_prefix.py [--requests 16] [--steps 8] [--bits 4] ...

A synthetic context is encoded, decoded straight into the blocks of slot 0 of
a paged cache, and forked to one slot per request: the requests share the
context's full blocks and own a copy of its last, partly filled one.  Each
decode step stores a new token's K and V in every request's blocks and attends
at every layer, the shared blocks read once for the batch.  Then every second
request ends, its blocks go back, the rest are compacted, and the others go on
with the same tables.  With --bits 4 or 8 the pool holds codes: the context is
quantised as it is put there, and so is every new token.  Queries, keys and
values of the new tokens are random: no model weights are involved.
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from kv_cache_compression_decode_gb300 import codec, paged, synth  # noqa: E402


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


def store_tokens(cache, slots, kv):
    """Append one token to each slot: kv [L][R][2][C] at the end of its blocks."""
    if isinstance(cache, paged.QuantCache):
        cache.lens[slots] += 1
        cache.write(kv[:, :, 0], kv[:, :, 1], slots=slots.int())
        return
    at = cache.lens[slots].long()
    block = cache.tables[slots, at // cache.block_tokens].long()
    cache.pool[:, block, :, at % cache.block_tokens] = kv.permute(1, 0, 2, 3)
    cache.lens[slots] += 1


def decode_step(cache, slots, shared_blocks, kv_heads, q_heads, head_dim, g):
    """One token for every request in `slots`; returns the outputs by layer."""
    L, C = cache.pool.shape[0], kv_heads * head_dim
    R = slots.shape[0]
    store_tokens(cache, slots.long(), torch.randn((L, R, 2, C), generator=g, device="cuda").half())
    q = torch.randn((L, R, 1, q_heads, head_dim), generator=g, device="cuda").half()
    out = [cache.attend(l, q[l], slots=slots, shared_slot=0, shared_blocks=shared_blocks) for l in range(L)]
    return q, torch.stack(out)


def run(layers=4, context=2000, kv_heads=8, q_heads=64, head_dim=128, block_tokens=16, requests=16, steps=8, seed=0,
        bits=16, log=print):
    C = kv_heads * head_dim
    cfg = codec.Config(layers, context, C)
    enc = codec.encode(cfg, synth.ar1_kv(layers, context, C, 0.95, 2, seed, device="cuda"))

    blocks = -(-context // block_tokens)
    own = -(-2 * steps // block_tokens) + 1
    size = layers, blocks + requests * own + 8, block_tokens
    if bits == 16:
        cache = paged.PagedCache.empty(*size, C, requests + 1, blocks + own)
    else:
        cache = paged.QuantCache.empty(*size, kv_heads, head_dim, requests + 1, blocks + own, bits)
    cache.fork(ints([paged.NO_SLOT]), ints([0]), ints([context]))  # blocks for the context
    cache.decode(cfg, enc, 0)
    slots = ints(range(1, requests + 1))
    cache.fork(ints([0] * requests), slots, ints([2 * steps] * requests))
    shared = context // block_tokens
    log(f"{requests} requests on a context of {context} tokens: {shared} blocks shared, "
        f"{int((cache.refs > 0).sum())} of {cache.refs.numel()} blocks in use")

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for _ in range(steps):
        q, out = decode_step(cache, slots, shared, kv_heads, q_heads, head_dim, g)
    cache.check()

    cache.free(slots[::2].contiguous())
    slots = slots[1::2].contiguous()
    cache.compact()
    for _ in range(steps):
        q, out = decode_step(cache, slots, shared, kv_heads, q_heads, head_dim, g)
    cache.check()
    used = int((cache.refs > 0).sum())
    log(f"{slots.shape[0]} requests left after {2 * steps} steps, {used} blocks in use at the front of the pool")
    return cache, slots, q, out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 4), ("context", 2000), ("kv-heads", 8), ("q-heads", 64), ("head-dim", 128),
                        ("block-tokens", 16), ("requests", 16), ("steps", 8), ("seed", 0), ("bits", 16)):
        ap.add_argument("--" + name, type=int, default=value)
    run(**vars(ap.parse_args()))
