"""More tiles for a block than 16 bits count."""

import pytest
import torch

from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_ten_million_tiles(cuda_ok):
    """170 sequences of one token, which sees its own key: out is v, dv is dout, and dq and dk are nothing but the
    difference of two sums of eight products."""
    import __graft_entry__
    __graft_entry__.build()
    n, heads, dim = 170, 65535, 8  # 11 million tiles, 73000 of a block
    gen = torch.Generator(device="cuda")
    gen.manual_seed(51)
    q, k, v, dout = (torch.randn(n, heads, dim, generator=gen, device="cuda", dtype=BF16) for _ in range(4))
    out, dq, dk, dv = (torch.full_like(q, 7.0) for _ in range(4))
    lse, at = torch.empty(n, heads, device="cuda"), torch.arange(n + 1, dtype=torch.int32, device="cuda")
    block = t.tpo_block_create(max(f(n, n, heads, heads, dim)
                                   for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace)))
    try:
        t.tpo_attention(block, q, k, v, out, q_start=at, lse=lse)
        assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
        t.tpo_attention_bwd(block, dout, q, k, v, out, lse, dq, dk, dv, q_start=at)
        assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    finally:
        t.tpo_block_destroy(block)
    assert torch.equal(out, v)
    want = (q.double() * k.double()).sum(2) * dim ** -0.5
    size = (q.double() * k.double()).abs().sum(2)
    assert ((lse.double() - want).abs() <= 32 * 2.0 ** -24 * (size + 1)).all()
    assert torch.equal(dv, dout)  # the weight is 1 but for some 2^-20
    slack = 64 * 2.0 ** -24 * (dout.double() * v.double()).abs().sum(2, keepdim=True)
    for g, x in ((dq, k), (dk, q)):
        assert (g.double().abs() <= 2 * slack * x.double().abs() + 2.0 ** -100).all()
