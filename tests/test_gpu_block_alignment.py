"""The block operators with vector arguments at every element offset: slices of
packed vectors, which need no more than their element's alignment."""

import pytest
import torch

import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def block(_built):
    b = t.tpo_block_create(max(t.tpo_block_workspace(t.TPO_OP_LINEAR_BWD, 1100, 1032, 520),
                               t.tpo_block_workspace(t.TPO_OP_LAYER_NORM_BWD, 20000, 20001)))
    yield b
    assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
    t.tpo_block_destroy(b)


@pytest.fixture(params=["rule", "pairs", "clusters", "clusters of 8"])
def any_path(request, block):
    t.tpo_block_set_opt(block, "path", dict(rule=0, pairs=1).get(request.param, 2))
    t.tpo_block_set_opt(block, "split", 8 if request.param.endswith("8") else 0)
    yield block
    t.tpo_block_set_opt(block, "path", 0)
    t.tpo_block_set_opt(block, "split", 0)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def d(v):
    return None if v is None else v.double()


def offset(v, by):
    """v as a slice that starts `by` elements into a packed vector of NaN."""
    buf = torch.full((v.numel() + by + 9,), float("nan"), dtype=v.dtype, device="cuda")
    buf[by:by + v.numel()] = v
    return buf[by:by + v.numel()]


@pytest.mark.parametrize("by", range(8))
@pytest.mark.parametrize("n,k,m", [(1, 264, 520), (5, 512, 7), (70, 136, 257), (130, 256, 384), (600, 200, 328)])
def test_bias(any_path, block, n, k, m, by):
    g = gen_of(10 * n + by)
    x, w, bias, res = rnd(g, n, k), rnd(g, m, k, scale=k ** -0.5), rnd(g, m), rnd(g, n, m)
    pitch = -(-m // 8) * 8
    y, z, r = (torch.zeros(n, pitch, dtype=BF16, device="cuda")[:, :m] for _ in range(3))
    r.copy_(res)
    t.tpo_linear(block, x, w, y, bias=offset(bias, by), act=t.TPO_ACT_GELU_TANH, residual=r, z=z)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.linear(d(x), d(w), d(bias), "gelu_tanh", d(res))
    R.check("y", y, want["y"])
    R.check("z", z, want["z"])


class Packed:
    """An output vector `by` elements into a packed one, whose other elements must stay as they are."""

    def __init__(self, count, dtype, by):
        self.buf = torch.full((count + by + 9,), GUARD, dtype=dtype, device="cuda")
        self.t = self.buf[by:by + count]
        self.t.fill_(float("nan"))
        self.by, self.count = by, count

    def get(self):
        rest = self.buf.clone()
        rest[self.by:self.by + self.count] = GUARD
        assert (rest == GUARD).all(), "written outside the output"
        return self.t


@pytest.mark.parametrize("by", range(1, 8))
@pytest.mark.parametrize("n,k,m", [(1, 264, 520), (70, 136, 257), (600, 200, 328)])
def test_bias_gradient(any_path, block, n, k, m, by):
    g = gen_of(20 * n + by)
    pitch = -(-m // 8) * 8
    dy, z = (torch.zeros(n, pitch, dtype=BF16, device="cuda")[:, :m] for _ in range(2))
    dy.copy_(rnd(g, n, m))
    z.copy_(rnd(g, n, m))
    x, w, db = rnd(g, n, k), rnd(g, m, k, scale=m ** -0.5), Packed(m, BF16, by)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    t.tpo_linear_bwd(block, dy, x, w, dx=dx, dw=dw, db=db.t, act=t.TPO_ACT_SILU, z=z)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.linear_bwd(d(dy), d(x), d(w), d(z), "silu")
    for name, v in (("dx", dx), ("dw", dw), ("db", db.get())):
        R.check(name, v, want[name])


# one and few rows, many rows of each of the kernels' forms, short rows, rows longer than a block holds
@pytest.mark.parametrize("n,k", [(1, 512), (3, 4096), (700, 1024), (1100, 4096), (400, 8192), (11000, 64), (3, 40000)])
@pytest.mark.parametrize("dt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("by", [(1, 0), (0, 3), (2, 4), (7, 5)])
def test_norm_weights(block, n, k, dt, wt, by):
    """Aligned rows; gamma and its gradient `by[0]` elements off, beta and its gradient, mean and rstd `by[1]`."""
    g = gen_of(n + k + 10 * by[0] + by[1])
    x, dy, dres = rnd(g, n, k, dtype=dt, scale=2) + 1.0, rnd(g, n, k, dtype=dt), rnd(g, n, k, dtype=dt)
    gamma, beta = rnd(g, k, dtype=wt), rnd(g, k, dtype=wt)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = Packed(n, F32, by[1]), Packed(n, F32, by[1])
    t.tpo_layer_norm(block, x, offset(gamma, by[0]), offset(beta, by[1]), y, mean=mean.t, rstd=rstd.t)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.layer_norm(d(x), d(gamma), d(beta), 1e-5)
    for name, v in (("y", y), ("mean", mean.get()), ("rstd", rstd.get())):
        R.check(name, v, want[name])
    dg, db = Packed(k, wt, by[0]), Packed(k, wt, by[1])
    t.tpo_layer_norm_bwd(block, dy, x, offset(gamma, by[0]), mean.t, rstd.t, dx, dgamma=dg.t, dbeta=db.t, dres=dres)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean.t), d(rstd.t), d(dres))
    for name, v in (("dx", dx), ("dgamma", dg.get()), ("dbeta", db.get())):
        R.check(name, v, want[name])
