"""Every key once, every query once: attention and its gradient on inputs whose
results are counts (attn_marks), over cuts, joins, caches and odd lengths."""

import pytest
import torch

import attn_marks as M
from tensor_comm_gemm_gb300 import tpoverlap as t

BF16 = torch.bfloat16
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def block(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()
    b = t.tpo_block_create(max(f(1 << 16, 1 << 17, 32, 16, 128)
                               for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace)))
    yield b
    t.tpo_block_destroy(b)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def synced(block):
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()


class Batch:
    """Queries lens[i] over klens[i] keys, packed or in a cache of so many rows a sequence."""

    def __init__(self, lens, klens, heads, kv, cache=0, device="cuda"):
        self.lens, self.klens, self.heads, self.kv = lens, klens, heads, kv
        q = torch.tensor([0] + lens).cumsum(0).tolist()
        k = [i * cache for i in range(len(lens))] if cache else torch.tensor([0] + klens).cumsum(0).tolist()
        self.n, self.nk, self.q_at, self.k_at = q[-1], cache * len(lens) if cache else k[-1], q, k
        self.q_in = torch.cat([torch.arange(c) for c in lens]).to(device)  # rows' places in their sequences
        self.q_of = torch.repeat_interleave(torch.tensor(lens), torch.tensor(lens)).to(device)
        self.k_of_q = torch.repeat_interleave(torch.tensor(klens), torch.tensor(lens)).to(device)
        self.k_in = torch.full((self.nk,), -1, device=device)
        for a, c in zip(k, klens):
            self.k_in[a:a + c] = torch.arange(c, device=device)

    def limit(self, causal):
        """Keys that each query sees."""
        return torch.clamp(self.q_in + 1 + self.k_of_q - self.q_of, min=0) if causal else self.k_of_q

    def where(self):
        if len(self.k_at) == len(self.lens):
            return dict(q_start=ints(self.q_at), k_start=ints(self.k_at), k_len=ints(self.klens))
        return dict(q_start=ints(self.q_at), k_start=ints(self.k_at))


def zeros(*shape):
    return torch.zeros(*shape, dtype=BF16, device="cuda")


CASES = [  # queries, keys, heads, key heads, dim, cache
    ([1], [33545], 8, 1, 128, 40960), ([2], [20001], 4, 4, 64, 0), ([1] * 64, [17 + 97 * ((i * 37) % 64) for i in range(64)], 8, 2, 64, 6200),
    ([300], [9000], 4, 1, 128, 0), ([512], [25088], 8, 1, 128, 0), ([2500], [2500], 2, 1, 64, 0),
    ([3001], [3001], 3, 3, 40, 0), ([2100, 5, 0, 900], [2100, 5, 7, 900], 6, 2, 80, 0), ([700, 129], [300, 1200], 5, 1, 96, 1300),
    ([4096], [4096], 8, 2, 128, 0), ([1] * 700, [7] * 700, 1, 1, 64, 0), ([40] * 9, [257] * 9, 32, 1, 24, 0),
]


@gpu
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both ways"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_each_key_counts_once(block, i, causal):
    lens, klens, heads, kv, dim, cache = CASES[i]
    torch.manual_seed(31)
    b = Batch(lens, klens, heads, kv, cache)
    limit = b.limit(causal)
    m = M.period(max(klens), dim)
    q, k = zeros(b.n, heads, dim), torch.randn(b.nk, kv, dim, device="cuda").to(BF16)
    k[b.k_in < 0] = float("nan")  # rows of the cache that are not in use
    out, lse = torch.empty_like(q), torch.empty(b.n, heads, device="cuda")
    for offset in range(0, m, dim):
        v = M.marks(b.k_in, dim, m, offset)[:, None].repeat(1, kv, 1)
        v[b.k_in < 0] = float("nan")
        t.tpo_attention(block, q, k, v, out, causal=causal, lse=lse, **b.where())
        synced(block)
        for h in range(heads):
            M.check_mean(out[:, h], lse[:, h], limit, dim, m, offset)


@gpu
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "both ways"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_each_pair_counts_once_in_the_gradients(block, i, causal):
    """p = 1 (q or k is 0, and so is lse); counts up to 256 are exact in bf16."""
    lens, klens, heads, kv, dim, cache = CASES[i]
    torch.manual_seed(31)
    b = Batch(lens, klens, heads, kv, cache)
    limit, group = b.limit(causal), heads // kv
    used = b.k_in >= 0
    # the queries that see a key: from this one on, of each of the group's heads
    of = [torch.full((b.nk,), 0, device="cuda") for _ in range(2)]
    for a, nq, nk in zip(b.k_at, lens, klens):
        of[0][a:a + nk], of[1][a:a + nk] = nq, nk
    first = torch.clamp(b.k_in - of[1] + of[0], min=0) if causal else 0 * b.k_in
    lse, out = torch.zeros(b.n, heads, device="cuda"), zeros(b.n, heads, dim)
    ones, ones_k = zeros(b.n, heads, dim), zeros(b.nk, kv, dim)
    ones[..., 0], ones_k[..., 0] = 1, 1
    none, none_k = zeros(b.n, heads, dim), zeros(b.nk, kv, dim)
    dq, dk, dv = zeros(b.n, heads, dim), zeros(b.nk, kv, dim), zeros(b.nk, kv, dim)
    rows = dict(q_rows=(max(lens) * group, b.q_in), k_rows=(max(klens), b.k_in))

    def call(dout, q, k, v):
        for g in (dq, dk, dv):
            g.fill_(7)
        t.tpo_attention_bwd(block, dout, q, k, v, out, lse, dq, dk, dv, causal=causal, scale=1.0, **b.where())
        synced(block)
        assert (dk[~used] == 7).all() and (dv[~used] == 7).all()

    m = M.period(rows["q_rows"][0], dim)
    of_keys = [M.below(of[0], dim, m, o) - M.below(first, dim, m, o) for o in range(0, m, dim)]
    for want, offset in zip(of_keys, range(0, m, dim)):
        want = (group * want[:, None]).repeat(1, kv, 1)[used]
        assert want.max() <= 256
        mark = M.marks(b.q_in, dim, m, offset)[:, None].repeat(1, heads, 1)
        call(mark, none, torch.randn(b.nk, kv, dim, device="cuda").to(BF16), none_k)
        assert torch.equal(dv[used].double(), want.double()) and not dk[used].any() and not dq.any()
        call(ones, mark, none_k, ones_k)  # ds = 1
        assert torch.equal(dk[used].double(), want.double()) and not dq.any()
    m = M.period(max(klens), dim)
    for offset in range(0, m, dim):
        mark = M.marks(b.k_in, dim, m, offset)[:, None].repeat(1, kv, 1)
        call(ones, none, mark, ones_k)
        want = M.below(limit, dim, m, offset)[:, None].repeat(1, heads, 1)
        assert torch.equal(dq.double(), want.double()) and not dk[used].any()


@pytest.mark.parametrize("keys", [1, 40, 700, 4000, 33545, 120000])
@pytest.mark.parametrize("dim", [24, 128])
def test_one_key_more_or_less_is_seen(keys, dim):
    """Results in the call's own types, of one key left out, one taken twice and one from behind the last."""
    m = M.period(keys, dim)
    at = torch.arange(keys + 1)

    def results(index, offset):
        count = M.marks(index, dim, m, offset, torch.float64).sum(0)
        return (count / len(index)).to(BF16)[None], torch.log(torch.tensor([float(len(index))]))

    limit, seen = torch.tensor([keys]), 0
    planted = {"left out": torch.cat([at[:keys // 2], at[keys // 2 + 1:keys]]), "one behind": at,
               "twice": torch.cat([at[:keys], at[keys // 3:keys // 3 + 1]]),
               "another's": torch.cat([at[:keys // 2], at[keys // 3:keys // 3 + 1], at[keys // 2 + 1:keys]])}
    for offset in range(0, m, dim):
        M.check_mean(*results(at[:keys], offset), limit, dim, m, offset)
    for name, index in planted.items():
        if not len(index) or torch.equal(index, at[:keys]):
            continue
        seen = 0
        for offset in range(0, m, dim):
            try:
                M.check_mean(*results(index, offset), limit, dim, m, offset)
            except AssertionError:
                seen += 1
        assert seen, name
