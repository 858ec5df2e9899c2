"""Values that are not finite reach the rows of the forward call that see their
key, and no others, whichever way the key is reached: each of the steps that
only some of a tile's rows see, whole and divided tiles, steps taken by turns."""

import pytest
import torch

from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def block(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    b = t.tpo_block_create(t.tpo_attention_workspace(1 << 14, 1 << 14, 8, 1, 128))
    yield b
    t.tpo_block_destroy(b)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dim", [40, 64, 128])
@pytest.mark.parametrize("heads,kv", [(4, 1), (2, 2), (3, 1)])
@pytest.mark.parametrize("nq,nk", [(3000, 3000), (3, 5000), (100, 4321), (300, 1111), (260, 260), (700, 690), (1, 129)])
def test_values_of_keys_reach_the_queries_that_see_them(block, nq, nk, heads, kv, dim, bad):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(nq + nk + dim)
    q, k, v = (torch.randn(r, h, dim, generator=gen, device="cuda").to(BF16) for r, h in ((nq, heads), (nk, kv), (nk, kv)))
    clean, out = torch.empty_like(q), torch.empty_like(q)
    lse, lse2 = (torch.empty(nq, heads, device="cuda") for _ in range(2))
    t.tpo_attention(block, q, k, v, clean, lse=lse)
    group = heads // kv
    tile = 256 // group if group != 3 else 84  # tokens of a tile
    limit = torch.arange(nq, device="cuda") + 1 + nk - nq
    firsts = sorted({0, tile * (nq // tile // 2), tile * (nq // tile)})
    for first in firsts:  # a tile's first token
        seen = max(0, first + 1 + nk - nq)
        keys = [x for x in (seen - 1, seen, seen + 127, seen + 128, seen + 255, nk - 1) if 0 <= x < nk]
        dirty, hit = v.clone(), torch.zeros_like(out, dtype=torch.bool)
        for i, key in enumerate(keys):  # each in a column of its own
            col, head = (7 * i + 3) % dim, i % kv
            dirty[key, head, col] = bad
            hit[limit > key, head * group:(head + 1) * group, col] = True
        out.fill_(0)
        t.tpo_attention(block, q, k, dirty, out, lse=lse2)
        assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
        assert not torch.isfinite(out[hit]).any(), (first, keys)
        assert torch.equal(out[~hit].view(torch.int16), clean[~hit].view(torch.int16)), (first, keys)
        assert torch.equal(lse, lse2)
