"""The attention sublayer's operators at their limits: more steps than a launch
can count, waits that run out, tensors past 32-bit offsets, many sequences,
captured gradients and graphs that share a workspace."""

import pytest
import torch

import attn_ref as A
import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def block(_built):
    b = t.tpo_block_create(max(f(1 << 16, 1 << 17, 128, 64, 128)
                               for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace)))
    yield b
    assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
    t.tpo_block_destroy(b)
    torch.cuda.empty_cache()


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def synced(block):
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()


def test_more_steps_than_are_counted(block):
    """2^18 sequences of a token over the same 2^20 keys are 2^31 steps."""
    batch, nk = 1 << 18, 1 << 20
    g = gen_of(1)
    q, k, v = rnd(g, batch, 1, 8), rnd(g, nk, 1, 8), rnd(g, nk, 1, 8)
    out = torch.full_like(q, 7.0)
    at = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    start = torch.zeros(batch, dtype=torch.int32, device="cuda")
    t.tpo_attention(block, q, k, v, out, q_start=at, k_start=start, k_len=torch.full_like(start, nk))
    assert t.tpo_block_sync_status(block) == t.TPO_ERR_UNSUPPORTED
    assert "2^31" in t.tpo_last_error()
    synced(block)
    assert (out == 7.0).all()
    lens = torch.full_like(start, 3)  # the handle goes on
    t.tpo_attention(block, q, k, v, out, q_start=at, k_start=start, k_len=lens)
    synced(block)
    some = q[:100]
    want = A.attention(some.double(), k[:3].double(), v[:3].double(), [(i, 1, 0, 3) for i in range(100)], True,
                       8 ** -0.5)
    R.check("out", out[:100], want["out"])
    last = A.attention(q[-1:].double(), k[:3].double(), v[:3].double(), [(0, 1, 0, 3)], True, 8 ** -0.5)
    R.check("out", out[-1:], last["out"])


def test_a_sequence_of_more_steps_than_are_counted(block):
    """2^24 tokens that all see 2^24 keys: 2^33 steps, in one of two sequences."""
    n = 1 << 24
    q, k, v, dout = (torch.zeros(n, 1, 8, dtype=BF16, device="cuda") for _ in range(4))
    out, dq, dk, dv = (torch.full_like(q, 7.0) for _ in range(4))
    lse, at = torch.full((n, 1), 7.0, device="cuda"), ints([0, n, n])
    mine = t.tpo_block_create(t.tpo_attention_bwd_workspace(n, n, 1, 1, 8))
    try:
        t.tpo_attention(mine, q, k, v, out, q_start=at, causal=False, lse=lse)
        assert t.tpo_block_sync_status(mine) == t.TPO_ERR_UNSUPPORTED
        t.tpo_attention_bwd(mine, dout, q, k, v, out, lse, dq, dk, dv, q_start=at, causal=False)
        assert t.tpo_block_sync_status(mine) == t.TPO_ERR_UNSUPPORTED
        synced(mine)
    finally:
        t.tpo_block_destroy(mine)
    assert all((x == 7.0).all() for x in (out, lse, dq, dk, dv))


def test_wait_that_runs_out_is_reported_once(block):
    """Parts of thousands of steps keep what writes them waiting for milliseconds: with a bound of one it gives up, with
    products and loads in flight, and a gradient behind it on the stream (whose own waits are all short) does too."""
    heads, n, nk = 32, 256, 1 << 21
    g = gen_of(2)
    q, k, v, dout = rnd(g, n, heads, 8), rnd(g, nk, heads, 8), rnd(g, nk, heads, 8), rnd(g, n, heads, 8)
    outs = [torch.empty_like(q), torch.empty(n, heads, device="cuda"), *(torch.empty_like(x) for x in (q, k, v))]

    def run():
        t.tpo_attention(block, q, k, v, outs[0], causal=False, lse=outs[1])
        t.tpo_attention_bwd(block, dout, q, k, v, *outs, causal=False)

    run()
    synced(block)
    first = [o.clone() for o in outs]
    assert all(torch.isfinite(o).all() for o in first)
    for _ in range(4):
        t.tpo_block_set_opt(block, "wait_timeout_ms", 1)
        run()
        assert t.tpo_block_sync_status(block) == 4
        assert "timed out" in t.tpo_last_error()
        synced(block)
        t.tpo_block_set_opt(block, "wait_timeout_ms", 2000)
        for o in outs:
            o.zero_()
        run()
        synced(block)
        assert all(torch.equal(o, f) for o, f in zip(outs, first))


def far(rows, heads, dim, ld):
    """[rows, heads, dim] whose last rows lie past 2^32 elements."""
    assert (rows - 1) * ld > 1 << 32
    buf = torch.empty((rows - 1) * ld + heads * dim, dtype=BF16, device="cuda")
    return buf.as_strided((rows, heads, dim), (ld, dim, 1))


def test_offsets_past_32_bits(block):
    g = gen_of(3)
    heads, kv, dim, rows, ld = 4, 2, 128, 2200, 1 << 21
    seqs = ((0, 100), (1900, 300))  # rows that are used
    q, dout = rnd(g, 400, heads, dim), rnd(g, 400, heads, dim)
    k, v = rnd(g, 400, kv, dim), rnd(g, 400, kv, dim)
    packed = ints([0, 100, 400])

    def run(q, k, v, dout, out, lse, dq, dk, dv, starts):
        t.tpo_attention(block, q, k, v, out, lse=lse, **starts)
        t.tpo_attention_bwd(block, dout, q, k, v, out, lse, dq, dk, dv, **starts)
        synced(block)

    near = [torch.empty_like(x) for x in (q, q, k, v)]
    run(q, k, v, dout, near[0], torch.empty(400, heads, device="cuda"), *near[1:], dict(q_start=packed))
    # the same with the second sequence far from the first: keys by start and length, queries as one more sequence of
    # which the rows between are empty of keys
    q_at, k_at, k_len = ints([0, 100, 1900, 2200]), ints([0, 0, 1900]), ints([100, 0, 300])
    there = [far(rows, heads if i in (0, 3, 4, 5) else kv, dim, ld) for i in range(8)]
    fq, fk, fv, fdout, fout, fdq, fdk, fdv = there
    where = torch.cat([torch.arange(a, a + c) for a, c in seqs]).cuda()
    for x, y in ((fq, q), (fk, k), (fv, v), (fdout, dout)):
        x[:] = 0
        x[where] = y
    run(fq, fk, fv, fdout, fout, torch.empty(rows, heads, device="cuda"), fdq, fdk, fdv,
        dict(q_start=q_at, k_start=k_at, k_len=k_len))
    for name, x, y in (("out", fout, near[0]), ("dq", fdq, near[1]), ("dk", fdk, near[2]), ("dv", fdv, near[3])):
        x = x[where].float()
        # the shares differ, so that sums may be cut elsewhere: each side is a rounding or two from the other
        assert ((x - y.float()).abs() <= 2.0 ** -7 * y.float().abs() + 2.0 ** -7 * y.float().abs().max()).all(), name
    assert (fout[100:1900] == 0).all()  # queries without keys
    del there, fq, fk, fv, fdout, fdq, fdk, fdv
    table = t.tpo_rotary_table(dim, 10000.0).cuda()
    pos, to = ints([5, 9, 70000]), ints([0, 2199, 2100])
    x, y = rnd(g, 3, heads, dim), torch.empty(3, heads, dim, dtype=BF16, device="cuda")
    t.tpo_rotary(block, x, table, y, pos=pos)
    t.tpo_rotary(block, x, table, fout, pos=pos, rows=to)
    synced(block)
    assert torch.equal(fout[to.long()], y)


def test_many_sequences(block):
    """More sequences than a block has threads, of any length: each comes to what it comes to alone."""
    g = gen_of(4)
    cpu = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 9, (3000,), generator=cpu)
    lens[::97] = 200
    at = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)])
    n = int(at[-1])
    q, k, v, dout = rnd(g, n, 4, 64), rnd(g, n, 1, 64), rnd(g, n, 1, 64), rnd(g, n, 4, 64)
    lse = torch.empty(n, 4, device="cuda")
    out, dq, dk, dv = (torch.empty_like(x) for x in (q, q, k, v))
    t.tpo_attention(block, q, k, v, out, q_start=at.int().cuda(), lse=lse)
    t.tpo_attention_bwd(block, dout, q, k, v, out, lse, dq, dk, dv, q_start=at.int().cuda())
    synced(block)
    seqs = [(int(at[i]), int(lens[i])) * 2 for i in range(len(lens))]
    d = lambda x: x.double()  # noqa: E731
    want = A.attention(d(q), d(k), d(v), seqs, True, 0.125)
    R.check("out", out, want["out"])
    R.check("lse", lse, want["lse"])
    ref = A.attention_bwd(d(dout), d(q), d(k), d(v), d(out), d(lse), seqs, True, 0.125)
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        R.check(name, got, ref[name])


def test_captured_steps_share_a_workspace(block):
    """Two captured training steps on one handle, replayed in turns: each gives the bits of its eager call."""
    g = gen_of(5)
    steps = []
    for n, heads, kv, dim in ((700, 4, 2, 128), (1500, 2, 2, 64)):
        q, k, v, dout = rnd(g, n, heads, dim), rnd(g, n, kv, dim), rnd(g, n, kv, dim), rnd(g, n, heads, dim)
        made = [torch.empty_like(q), torch.empty(n, heads, device="cuda"), *(torch.empty_like(x) for x in (q, k, v))]

        def call(q=q, k=k, v=v, dout=dout, made=made):
            t.tpo_attention(block, q, k, v, made[0], lse=made[1])
            t.tpo_attention_bwd(block, dout, q, k, v, *made)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        want = [x.clone() for x in made]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        steps.append((graph, made, want, call))  # the call keeps the inputs
    for _ in range(3):
        for graph, made, *_ in steps:
            for x in made:
                x.zero_()
            graph.replay()
        synced(block)
        for _, made, want, _ in steps:
            assert all(torch.equal(x, y) for x, y in zip(made, want))
