"""The block operators' gradients as wholes: the size of their error beside the
result's, and where values that are not finite spread to."""

import math

import pytest
import torch

import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ACT = dict(none=t.TPO_ACT_NONE, relu=t.TPO_ACT_RELU, gelu=t.TPO_ACT_GELU, gelu_tanh=t.TPO_ACT_GELU_TANH,
           silu=t.TPO_ACT_SILU)
NAN, INF = float("nan"), float("inf")
# Rounding to bf16 moves a value by an error that is uniform over a unit in the
# last place, of variance unit^2 / 12; the unit is at most 2^-7 of the value.
# So the root of the mean square error of a result rounded once is at most
ONCE = 2.0 ** -7 / math.sqrt(12.0)
# of the result's size, and, where the operand behind it was rounded before, too,
# the two (independent) errors together
TWICE = math.sqrt(2.0) * ONCE


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def block(_built):
    b = t.tpo_block_create(max(t.tpo_block_workspace(t.TPO_OP_GATED_BWD, 1100, 1032, 1000),
                               t.tpo_block_workspace(t.TPO_OP_LAYER_NORM_BWD, 20000, 40000)))
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


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n,k,m", [(64, 520, 1000), (300, 264, 520), (1100, 1032, 392)])
def test_size_of_the_linear_gradients_error(any_path, block, act, n, k, m):
    g = gen_of(n)
    dy, x, w = rnd(g, n, m), rnd(g, n, k), rnd(g, m, k, scale=m ** -0.5)
    z = None if act == "none" else rnd(g, n, m, scale=1.5)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(m, dtype=BF16, device="cuda")
    t.tpo_linear_bwd(block, dy, x, w, dx=dx, dw=dw, db=db, act=ACT[act], z=z)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.linear_bwd(d(dy), d(x), d(w), d(z), act)
    bound = ONCE if act == "none" else TWICE
    assert off(dx, want["dx"][0]) <= bound
    assert off(dw, want["dw"][0]) <= bound
    assert off(db, want["db"][0]) <= ONCE  # summed before the rounding of dz


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n,k,m", [(64, 520, 1000), (300, 264, 520), (1100, 1032, 392)])
def test_size_of_the_gated_gradients_error(any_path, block, act, n, k, m):
    gen = gen_of(n + 1)
    dh, g, u = rnd(gen, n, m), rnd(gen, n, m, scale=1.5), rnd(gen, n, m)
    x, wg, wu = rnd(gen, n, k), rnd(gen, m, k, scale=m ** -0.5), rnd(gen, m, k, scale=m ** -0.5)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    t.tpo_gated_bwd(block, dh, g, u, x, wg, wu, dx=dx, dwg=dwg, dwu=dwu, act=ACT[act])
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.gated_bwd(d(dh), d(g), d(u), d(x), d(wg), d(wu), act)
    for name, v in (("dx", dx), ("dwg", dwg), ("dwu", dwu)):
        assert off(v, want[name][0]) <= TWICE, name


@pytest.mark.parametrize("n,k", [(70, 1000), (700, 4096), (400, 5003), (11000, 64), (3, 40000)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_size_of_the_norm_gradients_error(block, n, k, dt):
    g = gen_of(n + 2)
    x, dy, gamma, dres = rnd(g, n, k, dtype=dt), rnd(g, n, k, dtype=dt), rnd(g, k, dtype=dt), rnd(g, n, k, dtype=dt)
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db, dres=dres)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    for name, v in (("dx", dx), ("dgamma", dg), ("dbeta", db)):
        # fp32: the roundings of a chain of up to n / 152 + 200 terms, each of 2^-24 of a partial sum at random
        fp32 = 2.0 ** -24 * math.sqrt(n / 152 + 200)
        assert off(v, want[name][0]) <= (ONCE if dt == BF16 else fp32), name


# ------------------------------------------------------------------ not finite

def same(name, got, want):
    """As R.check, and infinities of the same sign in the same places."""
    R.check(name, got, want)
    inf = torch.isinf(want[0])
    assert (got.double()[inf] == want[0][inf]).all(), name


def grad_of(z, act):
    """act'(z), which at NaN is NaN wherever it depends on z."""
    return R.act_grad(z, act) if act == "none" else torch.where(torch.isnan(z), z, R.act_grad(z, act))


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n", [5, 300])
def test_not_finite_values_in_the_linear_gradients(any_path, block, act, n):
    g = gen_of(31)
    k, m = 136, 200
    dy, x, w = rnd(g, n, m), rnd(g, n, k), rnd(g, m, k, scale=0.1)
    z = None if act == "none" else rnd(g, n, m)
    dy[1, 3] = NAN
    dy[2, 199] = INF
    x[3, 5] = -INF
    x[0, 135] = NAN
    if z is not None:
        z[4, 7], z[4, 8], z[4, 9] = NAN, INF, -INF
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(m, dtype=BF16, device="cuda")
    t.tpo_linear_bwd(block, dy, x, w, dx=dx, dw=dw, db=db, act=ACT[act], z=z)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    dz = d(dy) if z is None else d(dy) * grad_of(d(z), act)
    exact = R.linear_bwd(dz, d(x), d(w))            # the values
    slack = R.linear_bwd(d(dy), d(x), d(w), d(z), act)  # how far finite ones may be off
    for name, v in (("dx", dx), ("dw", dw), ("db", db)):
        same(name, v, (exact[name][0], slack[name][1]))
    rows = [r for r in range(n) if r not in (1, 2, 4)]
    assert torch.isfinite(dx[rows]).all() and not torch.isfinite(dx[1]).any() and not torch.isfinite(dx[2]).any()
    # a column of dw and a row of it are all that x's and dz's values reach
    cols, feats = [c for c in range(k) if c not in (5, 135)], [f for f in range(m) if f not in (3, 199, 7, 8, 9)]
    assert torch.isfinite(dw[feats][:, cols]).all() and torch.isfinite(db[feats]).all()


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n", [5, 300])
def test_not_finite_values_in_the_gated_gradients(any_path, block, act, n):
    gen = gen_of(32)
    k, m = 136, 200
    dh, g, u = rnd(gen, n, m), rnd(gen, n, m), rnd(gen, n, m)
    x, wg, wu = rnd(gen, n, k), rnd(gen, m, k, scale=0.1), rnd(gen, m, k, scale=0.1)
    dh[1, 3] = NAN
    u[2, 4] = INF
    g[3, 6] = NAN
    x[0, 135] = -INF
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    t.tpo_gated_bwd(block, dh, g, u, x, wg, wu, dx=dx, dwg=dwg, dwu=dwu, act=ACT[act])
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    dg, du = d(dh) * d(u) * grad_of(d(g), act), d(dh) * R.act(d(g), act)
    # (bounds of finite values: dg of the identity is one, whatever g is)
    slack = R.gated_bwd(d(dh), torch.nan_to_num(d(g)) if act == "none" else d(g), d(u), d(x), d(wg), d(wu), act)
    for name, v, ref in (("dx", dx, dg @ d(wg) + du @ d(wu)), ("dwg", dwg, dg.T @ d(x)), ("dwu", dwu, du.T @ d(x))):
        same(name, v, (ref, slack[name][1]))
    rows = [r for r in range(n) if r not in (1, 2, 3)]
    assert torch.isfinite(dx[rows]).all() and not torch.isfinite(dx[1]).any()
    cols, feats = list(range(135)), [f for f in range(m) if f not in (3, 4, 6)]
    assert torch.isfinite(dwg[feats][:, cols]).all() and torch.isfinite(dwu[feats][:, cols]).all()


@pytest.mark.parametrize("n,k", [(5, 96), (6, 4096), (700, 4096), (400, 5003), (11000, 64), (6, 40000)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_not_finite_values_in_the_norm_gradients(block, n, k, dt):
    g = gen_of(33)
    x, dy, gamma, dres = rnd(g, n, k, dtype=dt), rnd(g, n, k, dtype=dt), rnd(g, k, dtype=dt), rnd(g, n, k, dtype=dt)
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    dy[1, 3] = NAN
    dy[2, 7] = INF
    x[3, k - 1] = NAN
    dres[4, 5] = -INF
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db, dres=dres)
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    for name, v in (("dx", dx), ("dgamma", dg), ("dbeta", db)):
        same(name, v, want[name])
    rows = [r for r in range(n) if r not in (1, 2, 3, 4)]
    assert torch.isfinite(dx[rows]).all() and int((~torch.isfinite(dx[4])).sum()) == 1
    assert int((~torch.isfinite(dg)).sum()) == 3 and int((~torch.isfinite(db)).sum()) == 2
