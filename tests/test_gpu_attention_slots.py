"""Attention over a batch with long runs of slots that have no queries, as a
captured call with a fixed number of slots has."""

import pytest
import torch

import attn_ref as A
import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HEADS, KV, DIM, COUNT = 4, 2, 64, 340


@pytest.fixture(scope="module")
def case(cuda_ok):
    """More tiles than blocks, so that a share has some on both sides of a run in the middle."""
    import __graft_entry__
    __graft_entry__.build()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    lens = torch.randint(1, 200, (COUNT,), generator=torch.Generator().manual_seed(22))
    n = int(lens.sum())
    q, k, v, dout = (torch.randn(n, h, DIM, generator=gen, device="cuda", dtype=BF16) for h in (HEADS, KV, KV, HEADS))
    at = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    seqs = [(int(a), int(c)) * 2 for a, c in zip(at, lens)]
    d = lambda x: x.double()  # noqa: E731
    want = A.attention(d(q), d(k), d(v), seqs, True, DIM ** -0.5)
    out, lse = want["out"][0].to(BF16), want["lse"][0].float()
    ref = A.attention_bwd(d(dout), d(q), d(k), d(v), d(out), d(lse), seqs, True, DIM ** -0.5)
    return lens, (q, k, v, dout), (out, lse), want, ref


@pytest.mark.parametrize("empty", [31, 32, 33, 40000, 1 << 20])
def test_slots_without_queries_between_sequences(case, empty):
    """The whole call takes well below the bound of 100 ms that its waits get, and so must the way past the run."""
    lens, (q, k, v, dout), (o, l), want, ref = case
    lens = torch.cat([lens[:COUNT // 2], torch.zeros(empty, dtype=torch.long), lens[COUNT // 2:]])
    starts = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).int().cuda()
    n = len(q)
    lse = torch.empty(n, HEADS, device="cuda")
    out, dq, dk, dv = (torch.empty_like(x) for x in (q, q, k, v))
    block = t.tpo_block_create(max(f(n, n, HEADS, KV, DIM)
                                   for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace)))
    try:
        t.tpo_block_set_opt(block, "wait_timeout_ms", 100)
        t.tpo_attention(block, q, k, v, out, q_start=starts, lse=lse)
        assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
        t.tpo_attention_bwd(block, dout, q, k, v, o, l, dq, dk, dv, q_start=starts)
        assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    finally:
        t.tpo_block_destroy(block)
    R.check("out", out, want["out"])
    R.check("lse", lse, want["lse"])
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, ref[name])
