"""Attention calls behind one whose wait ran out: they give up too, with their
loads already in flight, and nothing of theirs reaches what runs after them."""

import pytest
import torch

from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


class Step:
    """Attention, its gradient and a product on one handle."""

    def __init__(self, gen, block, n, heads, kv, dim, causal=True):
        self.block, self.causal = block, causal
        self.q, self.dout = rnd(gen, n, heads, dim), rnd(gen, n, heads, dim)
        self.k, self.v = rnd(gen, n, kv, dim), rnd(gen, n, kv, dim)
        self.w = rnd(gen, 256, heads * dim)
        self.outs = [torch.empty_like(self.q), torch.empty(n, heads, device="cuda"),
                     *(torch.empty_like(x) for x in (self.q, self.k, self.v)), torch.empty(n, 256, dtype=BF16, device="cuda")]

    def run(self):
        out, lse, dq, dk, dv, y = self.outs
        t.tpo_attention(self.block, self.q, self.k, self.v, out, lse=lse, causal=self.causal)
        t.tpo_attention_bwd(self.block, self.dout, self.q, self.k, self.v, out, lse, dq, dk, dv, causal=self.causal)
        t.tpo_linear(self.block, self.dout.flatten(1), self.w, y)


def test_calls_behind_a_failed_one_leave_nothing_in_flight():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(41)
    need = max(f(1 << 12, 1 << 21, 32, 32, 128) for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace))
    blocks = [t.tpo_block_create(need) for _ in range(2)]  # the second never fails
    try:
        # parts of thousands of steps, whose end is waited for longer than a millisecond
        q, k, v = rnd(gen, 256, 32, 8), rnd(gen, 1 << 21, 32, 8), rnd(gen, 1 << 21, 32, 8)
        out = torch.empty_like(q)
        sizes = ((37, 8, 1, 128), (1, 8, 8, 64), (300, 6, 2, 80), (700, 4, 4, 64), (1500, 8, 2, 128))
        mine, other = ([Step(gen, b, *s) for s in sizes] for b in blocks)
        want = []
        for step in mine + other:
            step.run()
            want.append([x.clone() for x in step.outs])
        for b in blocks:
            assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
        for _ in range(5):
            t.tpo_block_set_opt(blocks[0], "wait_timeout_ms", 1)
            t.tpo_attention(blocks[0], q, k, v, out, causal=False)
            for a, b in zip(mine, other):
                for _ in range(3):
                    a.run()
                    b.run()
            assert t.tpo_block_sync_status(blocks[0]) == 4
            assert t.tpo_block_sync_status(blocks[1]) == 0, t.tpo_last_error()
            for step, first in zip(other, want[len(mine):]):
                assert all(torch.equal(x, y) for x, y in zip(step.outs, first))
            t.tpo_block_set_opt(blocks[0], "wait_timeout_ms", 2000)
            for step, first in zip(mine, want):
                for x in step.outs:
                    x.zero_()
                step.run()
                assert t.tpo_block_sync_status(blocks[0]) == 0, t.tpo_last_error()
                assert all(torch.equal(x, y) for x, y in zip(step.outs, first))
    finally:
        for b in blocks:
            t.tpo_block_destroy(b)
