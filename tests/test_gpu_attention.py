"""The attention sublayer's operators on the GPU against their definitions in
64 bits (attn_ref): head layouts, lengths from none on, odd sizes, pitches,
rows that no sequence has, values that are not finite, other streams, graph
capture and repeated calls."""

import math

import pytest
import torch

import attn_ref as A
import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN = math.nan
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def block(_built):
    b = t.tpo_block_create(max(f(1 << 16, 1 << 17, 128, 64, 128)
                               for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace)))
    yield b
    assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
    t.tpo_block_destroy(b)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def synced(block):
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()


def framed(v, how):
    """v [rows, heads, dim] as a view of a larger buffer whose other elements are NaN: 'dense', 'fused' (between other
    heads), 'heads' (heads outermost) or 'wide' (gaps behind each head and row)."""
    if how == "dense":
        return v.clone()
    n, h, d = v.shape
    if how == "heads":
        buf = torch.full((h, n + 1, d), NAN, dtype=v.dtype, device="cuda")
        view = buf[:, :n].transpose(0, 1)
    elif how == "wide":
        buf = torch.full((n, h + 1, d + 8), NAN, dtype=v.dtype, device="cuda")
        view = buf[:, :h, :d]
    else:
        buf = torch.full((n, h + 3, d), NAN, dtype=v.dtype, device="cuda")
        view = buf[:, 1:h + 1]
    view.copy_(v)
    return view


class Out:
    """An output of v's shape in a frame; elements outside it and rows of no sequence must stay as they were."""

    def __init__(self, v, how, rows, dtype=None):
        self.t = framed(torch.full(v.shape, NAN, dtype=dtype or v.dtype, device="cuda"), how)
        self.base = self.t if self.t._base is None else self.t._base
        self.base.fill_(GUARD)
        self.rows = rows

    def get(self):
        rest = self.base.clone()
        view = rest.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset())
        view[self.rows] = GUARD
        assert (rest == GUARD).all(), "written outside the sequences' rows"
        return self.t


def rows_of(seqs, first, count):
    r = [torch.arange(s[first], s[first] + s[count]) for s in seqs]
    return torch.cat(r).cuda() if r else torch.empty(0, dtype=torch.long, device="cuda")


def layout(lens, klens, cache, behind=0):
    """(sequences, rows of q, rows of k, arguments) of packed queries over packed or cached keys."""
    seqs, q0, k0 = [], 0, 0
    for i, (nq, nk) in enumerate(zip(lens, klens)):
        seqs.append((q0, nq, i * cache if cache else k0, nk))
        q0, k0 = q0 + nq, k0 + nk
    kw = dict(q_start=ints([s[0] for s in seqs] + [q0]))
    if cache:
        kw.update(k_start=ints([s[2] for s in seqs]), k_len=ints(list(klens)))
    else:
        kw.update(k_start=ints([s[2] for s in seqs] + [k0]))
    return seqs, q0 + behind, (cache * len(lens) if cache else k0 + behind), kw


def run_case(block, lens, klens, heads, kv, dim, causal, cache=0, how="dense", behind=0, seed=1, scale=None, bwd=True,
             forward=True):
    g = gen_of(seed)
    seqs, n, nk, kw = layout(lens, klens, cache, behind)
    q, k, v = rnd(g, n, heads, dim), rnd(g, nk, kv, dim), rnd(g, nk, kv, dim)
    used_q, used_k = rows_of(seqs, 0, 1), rows_of(seqs, 2, 3)
    for x, used in ((q, used_q), (k, used_k), (v, used_k)):  # rows of no sequence
        keep = x[used].clone()
        x.fill_(NAN)
        x[used] = keep
    q, k, v = (framed(x, how) for x in (q, k, v))
    c = dim ** -0.5 if scale is None else scale
    d = lambda x: x.double()  # noqa: E731
    want = A.attention(d(q), d(k), d(v), seqs, causal, c)
    if forward:
        out, lse = Out(q, how, used_q), Out(torch.empty(n, heads, device="cuda"), "dense", used_q, F32)
        t.tpo_attention(block, q, k, v, out.t, causal=causal, scale=scale, lse=lse.t, **kw)
        synced(block)
        for name, got in (("out", out), ("lse", lse)):
            R.check(name, got.get()[used_q], tuple(x[used_q] for x in want[name]))
        again = Out(q, how, used_q)
        t.tpo_attention(block, q, k, v, again.t, causal=causal, scale=scale, **kw)  # without lse, the same bits
        synced(block)
        assert torch.equal(again.get().view(torch.int16), out.t.view(torch.int16))
    if not bwd:
        return
    dout = torch.full_like(q, NAN)
    dout[used_q] = rnd(g, len(used_q), heads, dim)
    out, lse = want["out"][0].to(BF16), want["lse"][0].float().contiguous()
    grads = {"d" + x: Out(y, how, u) for x, y, u in (("q", q, used_q), ("k", k, used_k), ("v", v, used_k))}
    dout, o = framed(dout, how), framed(out, how)
    t.tpo_attention_bwd(block, dout, q, k, v, o, lse, *(x.t for x in grads.values()), causal=causal, scale=scale, **kw)
    synced(block)
    ref = A.attention_bwd(d(dout), d(q), d(k), d(v), d(out), d(lse), seqs, causal, c)
    for name, got in grads.items():
        used = used_q if name == "dq" else used_k
        R.check(name, got.get()[used], tuple(x[used] for x in ref[name]))
    again = {x: Out(y.t, "dense", y.rows) for x, y in grads.items()}
    t.tpo_attention_bwd(block, dout, q, k, v, o, lse, *(x.t for x in again.values()), causal=causal, scale=scale, **kw)
    synced(block)
    for name in grads:
        assert torch.equal(again[name].t[again[name].rows], grads[name].t[again[name].rows]), name


HOWS = ("dense", "fused", "wide", "heads")
CASES = [  # heads, kv heads, dim, queries, keys (None: the same)
    (1, 1, 64, [1], None), (1, 1, 128, [2], None), (4, 4, 128, [128], None), (4, 1, 128, [128], [129]),
    (8, 1, 128, [37], None), (2, 2, 64, [127, 1, 129], None), (6, 2, 80, [65, 0, 200, 7], None),
    (8, 2, 128, [255, 257], None), (5, 1, 96, [100, 31], None), (7, 1, 128, [19, 300], None),
    (3, 3, 40, [33, 500], None), (16, 1, 128, [50, 9], None), (128, 1, 64, [3, 12], None), (9, 3, 8, [70], None),
    (4, 2, 128, [5, 0, 40, 300], [9, 3, 40, 10]), (4, 2, 64, [3, 4, 0], [0, 200, 0]), (2, 1, 128, [1, 1, 1], [1, 128, 513]),
    (8, 1, 128, [4, 2, 1], [1000, 255, 256]), (64, 8, 64, [1, 1], [300, 31]), (33, 1, 72, [17], [333]),
    (2, 1, 24, [700], None), (1, 1, 128, [513], [1100]),
]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both ways"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention_and_gradients(block, i, causal):
    heads, kv, dim, lens, klens = CASES[i]
    run_case(block, lens, klens or lens, heads, kv, dim, causal, how=HOWS[i % 4], behind=3 * (i % 2), seed=100 + i)


@pytest.mark.parametrize("how", HOWS)
def test_layouts(block, how):
    run_case(block, [90, 140], [90, 140], 6, 2, 64, True, how=how, behind=5, seed=3)


@pytest.mark.parametrize("few", [1, 3])
@pytest.mark.parametrize("heads,kv,dim", [(8, 1, 128), (8, 8, 64), (12, 2, 80)])
def test_tokens_over_a_cache(block, heads, kv, dim, few):
    klens = [few, 128, 1000, 17 + few, 777]
    for how in ("dense", "heads"):
        run_case(block, [few] * 5, klens, heads, kv, dim, True, cache=1024, how=how, seed=few, bwd=False)


@pytest.mark.parametrize("lens,klens,heads,kv,dim,causal", [
    ([1], [20000], 8, 1, 128, True),       # one token over a long cache: cut among the SMs
    ([1] * 40, list(range(1, 4001, 100)), 4, 2, 128, True),
    ([300], [9000], 4, 1, 128, True), ([2500], [2500], 2, 1, 64, True), ([2100, 5, 900], [2100, 5, 900], 3, 3, 128, False),
    ([1] * 700, [7] * 700, 1, 1, 64, True),  # more sequences than threads
])
def test_long(block, lens, klens, heads, kv, dim, causal):
    run_case(block, lens, klens, heads, kv, dim, causal, seed=11, bwd=max(klens) < 9000)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_scales(block, scale):
    run_case(block, [150, 20], [150, 20], 4, 2, 64, True, seed=12, scale=scale)


def test_one_sequence_needs_no_arrays(block):
    g = gen_of(13)
    q, k, v = rnd(g, 70, 4, 64), rnd(g, 200, 2, 64), rnd(g, 200, 2, 64)
    out = torch.empty_like(q)
    for kw, nk in ((dict(), 200), (dict(k_len=ints([77])), 77), (dict(k_start=ints([50]), k_len=ints([100])), 100)):
        t.tpo_attention(block, q, k, v, out, **kw)
        synced(block)
        want = A.attention(q.double(), k.double(), v.double(), [(0, 70, 50 if "k_start" in kw else 0, nk)], True, 0.125)
        R.check("out", out, want["out"])


def test_keys_lie_as_the_queries_do(block):
    g = gen_of(14)
    q, k, v = rnd(g, 90, 4, 64), rnd(g, 90, 2, 64), rnd(g, 90, 2, 64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    at = ints([0, 30, 90])
    t.tpo_attention(block, q, k, v, a, q_start=at)
    t.tpo_attention(block, q, k, v, b, q_start=at, k_start=at)
    synced(block)
    assert torch.equal(a, b)


def test_starts_and_lengths_are_held_inside_the_tensors(block):
    g = gen_of(15)
    q, k, v = rnd(g, 20, 2, 64), rnd(g, 30, 2, 64), rnd(g, 30, 2, 64)
    used = torch.arange(20, device="cuda")
    out = Out(q, "fused", used)
    # the second sequence's queries run past the end, its keys too; the third has a start behind the end
    t.tpo_attention(block, q, k, v, out.t, q_start=ints([-5, 8, 1 << 30, 2000000000]), k_start=ints([-7, 10, 99]),
                    k_len=ints([9, 1 << 30, 5]), causal=False)
    synced(block)
    want = A.attention(q.double(), k.double(), v.double(), [(0, 8, 0, 9), (8, 12, 10, 20)], False, 0.125)
    R.check("out", out.get(), want["out"])


def test_nothing_to_do(block):
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    k = rnd(gen_of(1), 9, 2, 64)
    t.tpo_attention(block, e, k, k, e)
    q, out = rnd(gen_of(2), 5, 2, 64), torch.ones(5, 2, 64, dtype=BF16, device="cuda")
    lse = torch.zeros(5, 2, device="cuda")
    t.tpo_attention(block, q, e, e, out, lse=lse)
    dk, dv = torch.ones_like(k), torch.ones_like(k)
    t.tpo_attention_bwd(block, e, e, k, k, e, torch.empty(0, 2, device="cuda"), e, dk, dv)
    dq = torch.ones_like(q)
    t.tpo_attention_bwd(block, q, q, e, e, out, lse, dq, e, e)
    t.tpo_attention_bwd(block, e, e, e, e, e, None, e, e, e)
    synced(block)
    assert not out.any() and (lse == -math.inf).all() and not dk.any() and not dv.any() and not dq.any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_not_finite_stay_where_they_belong(block, bad):
    """A key that a query does not see does not reach it, whatever it holds; a row of q reaches its own output only."""
    g = gen_of(16)
    lens, heads, kv, dim = [100, 150], 4, 2, 64
    seqs, n, nk, kw = layout(lens, lens, 0)
    q, k, v = rnd(g, n, heads, dim), rnd(g, nk, kv, dim), rnd(g, nk, kv, dim)
    clean = torch.empty_like(q)
    t.tpo_attention(block, q, k, v, clean, **kw)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    v2[60, 0, 5], k2[70, 1, 3], q2[120, 2, 1] = bad, bad, bad
    out = torch.empty_like(q)
    t.tpo_attention(block, q2, k2, v2, out, **kw)
    synced(block)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[60:100, 0:2, 5] = True   # the value's column, for the queries that see the key
    hit[70:100, 2:4] = True      # scores of NaN or of either infinity
    hit[120, 2] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert not torch.isfinite(out[60:100, 0:2, 5]).any()
    if math.isnan(bad):
        assert torch.isnan(out[70:100, 2:4]).all() and torch.isnan(out[120, 2]).all()


def test_gradients_of_other_sequences_stay_clean(block):
    """NaN in one sequence (and behind the last) does not reach another's gradients."""
    g = gen_of(17)
    lens, heads, kv, dim = [100, 90, 130], 4, 2, 64
    seqs, n, nk, kw = layout(lens, lens, 0, behind=4)
    q, k, v, dout = rnd(g, n, heads, dim), rnd(g, nk, kv, dim), rnd(g, nk, kv, dim), rnd(g, n, heads, dim)
    out, lse = torch.empty_like(q), torch.empty(n, heads, device="cuda")
    t.tpo_attention(block, q, k, v, out, lse=lse, **kw)
    clean, got = ([torch.zeros_like(x) for x in (q, k, v)] for _ in range(2))
    t.tpo_attention_bwd(block, dout, q, k, v, out, lse, *clean, **kw)
    for x in (q, k, v, dout, out, lse):
        x[100:190] = NAN
        x[320:] = NAN
    t.tpo_attention_bwd(block, dout, q, k, v, out, lse, *got, **kw)
    synced(block)
    for a, b in zip(clean, got):
        for r in (slice(0, 100), slice(190, 320)):
            assert torch.equal(a[r], b[r])
        assert not b[320:].any() and torch.isnan(b[100:190]).any()


def test_capture_follows_lengths_and_other_streams(block):
    g = gen_of(18)
    heads, kv, dim, cache = 8, 2, 128, 900
    q, k, v = rnd(g, 3, heads, dim), rnd(g, 3 * cache, kv, dim), rnd(g, 3 * cache, kv, dim)
    out, at, start, lens = torch.empty_like(q), ints([0, 1, 2, 3]), ints([0, cache, 2 * cache]), ints([1, 1, 1])
    call = lambda: t.tpo_attention(block, q, k, v, out, q_start=at, k_start=start, k_len=lens)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([1, 5, 900], [300, 129, 128], [0, 900, 17]):
        lens.copy_(ints(now))
        q.copy_(rnd(g, 3, heads, dim))
        graph.replay()
        synced(block)
        want = A.attention(q.double(), k.double(), v.double(), [(i, 1, i * cache, now[i]) for i in range(3)], True,
                           dim ** -0.5)
        R.check("out", out, want["out"])


def test_two_handles_on_two_streams():
    need = max(t.tpo_attention_workspace(600, 600, 8, 2, 128), t.tpo_attention_bwd_workspace(600, 600, 8, 2, 128))
    blocks = [t.tpo_block_create(need) for _ in range(2)]
    try:
        g = gen_of(19)
        q, k, v, dout = rnd(g, 600, 8, 128), rnd(g, 600, 2, 128), rnd(g, 600, 2, 128), rnd(g, 600, 8, 128)
        made = []
        for b in blocks:
            made.append([torch.empty_like(q), torch.empty(600, 8, device="cuda")] +
                        [torch.empty_like(x) for x in (q, k, v)])
        torch.cuda.synchronize()
        for b, o in zip(blocks, made):
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    t.tpo_attention(b, q, k, v, o[0], lse=o[1])
                    t.tpo_attention_bwd(b, dout, q, k, v, o[0], o[1], *o[2:])
        torch.cuda.synchronize()
        for b in blocks:
            assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
        for x, y in zip(*made):
            assert torch.equal(x, y)
    finally:
        for b in blocks:
            t.tpo_block_destroy(b)


# ------------------------------------------------------------------ rotary

ROTARY = [  # rows, heads, dim, rot
    (1, 1, 2, 2), (1, 40, 128, 128), (3, 5, 128, 64), (17, 9, 80, 32), (5, 3, 7, 6), (33, 2, 96, 48), (100, 1, 64, 64),
    (700, 3, 40, 20), (9, 72, 128, 128), (4, 2, 16, 0), (2, 3, 1, 0), (1500, 2, 64, 16), (2, 1, 1024, 1000),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pairs", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("n,heads,dim,rot", ROTARY)
def test_rotary(block, n, heads, dim, rot, pairs, dtype):
    i = ROTARY.index((n, heads, dim, rot))
    g = gen_of(200 + i)
    how = HOWS[i % 4]
    x = framed(rnd(g, n, heads, dim, dtype=dtype), how)
    table = t.tpo_rotary_table(rot, 10000.0).cuda()
    lay = t.TPO_ROTARY_PAIRS if pairs else t.TPO_ROTARY_HALVES
    pos = torch.randint(-100, 2 ** 31 - 1 if i % 2 else 5000, (n,), generator=g, device="cuda").to(torch.int32)
    used = torch.arange(n, device="cuda")
    for inverse, magnitude in ((False, 1.0), (True, 1.25)):
        want = A.rotary(x.double(), pos, A.frequencies(rot, 10000.0), pairs, inverse, magnitude)
        y = Out(x, how, used)
        t.tpo_rotary(block, x, table, y.t, pos=pos, layout=lay, inverse=inverse, magnitude=magnitude)
        synced(block)
        R.check("y", y.get(), want)
    z = x.clone()
    t.tpo_rotary(block, z, table, z, pos=pos, layout=lay, inverse=True, magnitude=1.25)  # in place
    # rows of another order in a larger buffer; some left out
    ny = n + 3
    rows = torch.randperm(ny, generator=g, device="cuda")[:n].to(torch.int32)
    if n > 2:
        rows[1], rows[2] = -1, ny
    kept = (rows >= 0) & (rows < ny)
    into = Out(torch.empty(ny, heads, dim, dtype=dtype, device="cuda"), how, rows[kept].long())
    t.tpo_rotary(block, x, table, into.t, pos=pos, layout=lay, inverse=True, magnitude=1.25, rows=rows)
    synced(block)
    assert torch.equal(z, y.t)
    assert torch.equal(into.get()[rows[kept].long()], y.t[kept])


def test_rotary_counts_rows_without_positions(block):
    x = rnd(gen_of(4), 300, 2, 64)
    table = t.tpo_rotary_table(64, 10000.0).cuda()
    y = torch.empty_like(x)
    t.tpo_rotary(block, x, table, y)
    synced(block)
    R.check("y", y, A.rotary(x.double(), torch.arange(300, device="cuda"), A.frequencies(64, 10000.0)))


@pytest.mark.parametrize("offset", [1, 2, 3, 4, 5])
def test_rotary_at_every_alignment(block, offset):
    g = gen_of(5)
    x = rnd(g, 40 * 3 * 32 + 8)[offset:offset + 40 * 3 * 32].view(40, 3, 32)
    table = t.tpo_rotary_table(32, 10000.0).cuda()
    y = torch.empty(40 * 3 * 32 + 8, dtype=BF16, device="cuda")[8 - offset:8 - offset + 40 * 3 * 32].view(40, 3, 32)
    t.tpo_rotary(block, x, table, y)
    synced(block)
    R.check("y", y, A.rotary(x.double(), torch.arange(40, device="cuda"), A.frequencies(32, 10000.0)))


def test_rotary_of_no_rows(block):
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    t.tpo_rotary(block, e, t.tpo_rotary_table(64).cuda(), e)
    synced(block)
