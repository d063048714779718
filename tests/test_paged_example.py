"""The example that runs the page calls and the attention together."""
import numpy as np
import pytest
import torch

from tests.test_paged_attend import check

needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


@pytest.mark.gpu
@needs_gpu
@pytest.mark.parametrize("context,requests,block_tokens", [(333, 6, 16), (320, 3, 32), (1000, 20, 64)])
def test_requests_continue_a_decoded_context(context, requests, block_tokens):
    """After 2 x 5 steps, a free and a compaction, the last step's outputs are
    the formula's over the tables as they are, the blocks in use are the first
    of the pool, and their references are those of the tables."""
    from examples import shared_prefix

    lines = []
    cache, slots, q, out = shared_prefix.run(layers=2, context=context, kv_heads=2, q_heads=8, head_dim=64,
                                             block_tokens=block_tokens, requests=requests, steps=5, log=lines.append)
    assert len(lines) == 2
    lens = cache.lens.tolist()
    assert [lens[s] for s in slots.tolist()] == [context + 10] * len(slots) and lens[0] == context
    for layer in range(2):
        lse = torch.empty(q[layer].shape[:3], device="cuda")
        again = cache.attend(layer, q[layer], slots=slots, shared_slot=0, shared_blocks=context // block_tokens, lse=lse)
        assert torch.equal(again, out[layer])
        check(cache, q[layer], out[layer], lse, slots, layer, 64 ** -0.5)
    tables, refs = cache.tables.cpu().numpy(), cache.refs.cpu().numpy()
    assert np.array_equal(np.bincount(tables[tables >= 0], minlength=len(refs)), refs)
    assert (refs[: (refs > 0).sum()] > 0).all()
