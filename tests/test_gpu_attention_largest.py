"""The attention sublayer's operators at the largest numbers of rows."""

import math

import pytest
import torch

import attn_ref as A
import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ROWS = 1 << 30


@pytest.fixture
def block(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    if torch.cuda.get_device_properties(0).total_memory < 150e9:
        pytest.skip("needs 150 GB")
    b = t.tpo_block_create(max(t.tpo_attention_workspace(ROWS, ROWS, 1, 1, 8),
                               t.tpo_attention_bwd_workspace(1 << 16, ROWS, 1, 1, 8)))
    yield b
    t.tpo_block_destroy(b)
    torch.cuda.empty_cache()


def synced(block):
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()


def rnd(*shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(71)
    return torch.randn(*shape, generator=gen, device="cuda").to(BF16)


def test_queries(block):
    """2^30 queries, the same 2^12 again and again, over 300 keys."""
    some = rnd(1 << 12, 1, 8)
    k, v = rnd(300, 1, 8), rnd(300, 1, 8).flip(0).contiguous()
    q, out = (torch.empty(ROWS, 1, 8, dtype=BF16, device="cuda") for _ in range(2))
    q.view(-1, *some.shape).copy_(some)
    lse = torch.empty(ROWS, 1, device="cuda")
    t.tpo_attention(block, q, k, v, out, causal=False, lse=lse)
    synced(block)
    want = A.attention(some.double(), k.double(), v.double(), [(0, len(some), 0, 300)], False, 8 ** -0.5)
    for name, got in (("out", out), ("lse", lse)):
        first = got[:len(some)]
        R.check(name, first, want[name])
        # a whole tile's bits are the same again; the few divided ones are checked
        bits = got.view(torch.int16 if name == "out" else torch.int32)
        other = (bits.view(-1, *first.shape) != bits[:len(some)]).flatten(2).any(2).flatten().nonzero().flatten()
        assert len(other) <= 152 * 256
        R.check(name, got[other], tuple(w[other % len(some)] for w in want[name]))


def test_keys(block):
    """A token over 2^30 keys, all of the same score: the sum counts them, and a marked key in 2^20 is a share of 2^-20;
    then the gradients, with a weight of one: each value gets the token's."""
    q, k = torch.zeros(1, 1, 8, dtype=BF16, device="cuda"), rnd(1, 1, 8).expand(ROWS, 1, 8).contiguous()
    v = torch.ones(ROWS, 1, 8, dtype=BF16, device="cuda")
    v[..., 1] = 0
    v.view(-1, 1 << 20, 8)[:, 12345, 1] = 1
    out, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    t.tpo_attention(block, q, k, v, out, lse=lse)
    synced(block)
    log = math.log(ROWS)
    assert abs(float(lse) - log) <= 4 * R.U32 * log
    want = torch.ones(8, dtype=torch.float64, device="cuda")
    want[1] = 2.0 ** -20
    assert ((out.double().view(8) - want).abs() <= (R.U16 + 160 * R.U32) * want).all()
    del v
    dout, dq = rnd(1, 1, 8), torch.empty_like(q)
    dk, dv = (torch.full_like(k, 7.0) for _ in range(2))
    zero = torch.zeros_like(lse)
    t.tpo_attention_bwd(block, dout, q, k, torch.zeros_like(k), torch.zeros_like(q), zero, dq, dk, dv)
    synced(block)
    assert (dv == dout).all() and not dk.any() and not dq.any()


def test_rotary_rows(block):
    x = rnd(1 << 16, 1, 2).repeat(ROWS >> 16, 1, 1)
    y, table = torch.full_like(x, 7.0), t.tpo_rotary_table(2).cuda()
    t.tpo_rotary(block, x, table, y)  # positions are the rows' numbers
    synced(block)
    for first in (0, ROWS // 2 - 5, ROWS - (1 << 16)):
        at = torch.arange(first, first + (1 << 16), device="cuda")
        R.check("y", y[at], A.rotary(x[at].double(), at, A.frequencies(2, 10000.0)))
    assert not (y == 7.0).all(2).any()
