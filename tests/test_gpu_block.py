"""The block operators on the GPU against their definitions in 64 bits
(block_ref): types, odd sizes, pitches, empty batches, values that are not
finite, buffers that alias where the contract allows it, other streams, graph
capture and repeated calls."""

import math

import pytest
import torch

import block_ref as R
from tensor_comm_gemm_gb300 import tpoverlap as t

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ACT = dict(none=t.TPO_ACT_NONE, relu=t.TPO_ACT_RELU, gelu=t.TPO_ACT_GELU, gelu_tanh=t.TPO_ACT_GELU_TANH,
           silu=t.TPO_ACT_SILU)
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def block(_built):
    b = t.tpo_block_create(max(t.tpo_block_workspace(t.TPO_OP_GATED_BWD, 4200, 4096, 4096),
                               t.tpo_block_workspace(t.TPO_OP_LAYER_NORM_BWD, 20000, 40000)))
    yield b
    assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
    t.tpo_block_destroy(b)


@pytest.fixture(params=["rule", "pairs", "clusters", "clusters of 8"])
def any_path(request, block):
    """Every form of the products, whatever the rule would take."""
    t.tpo_block_set_opt(block, "path", dict(rule=0, pairs=1).get(request.param, 2))
    t.tpo_block_set_opt(block, "split", 8 if request.param.endswith("8") else 0)
    yield block
    t.tpo_block_set_opt(block, "path", 0)
    t.tpo_block_set_opt(block, "split", 0)


def rnd(gen, *shape, dtype=BF16, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Out:
    """An output [n, m] inside a wider buffer whose other elements must stay as they are."""

    def __init__(self, n, m, dtype=BF16, unit=8, extra=1):
        pitch = -(-m // unit) * unit + extra * unit
        self.buf = torch.full((n + 2, pitch), GUARD, dtype=dtype, device="cuda")
        self.t = self.buf[1:n + 1, :m]
        self.t.fill_(float("nan"))
        self.n, self.m = n, m

    def get(self):
        rest = self.buf.clone()
        rest[1:self.n + 1, :self.m] = GUARD
        assert (rest == GUARD).all(), "written outside the output"
        return self.t


def pitched(v, unit, extra=0):
    """v as a view whose row pitch is a multiple of `unit` (plus `extra` units), NaN in between."""
    n, m = v.shape
    pitch = -(-m // unit) * unit + extra * unit
    if v.dtype == E4M3:
        buf = torch.full((n, pitch), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)  # NaN codes
        buf.view(torch.uint8)[:, :m] = v.view(torch.uint8)
    else:
        buf = torch.full((n, pitch), float("nan"), dtype=v.dtype, device="cuda")
        buf[:, :m] = v
    return buf[:, :m]


def d(v):
    return None if v is None else v.double()


def codes(v):
    inv = (v.float().abs().amax() / 448).reshape(1)
    return (v.float() / inv).to(E4M3), inv


def synced(block):
    assert t.tpo_block_sync_status(block) == 0, t.tpo_last_error()


# ------------------------------------------------------------------ linear

SHAPES = [  # n, k, m
    (1, 8, 8), (1, 1, 1), (1, 4096, 520), (2, 40, 1032), (3, 72, 40), (5, 9, 7), (8, 520, 2048), (16, 1000, 264),
    (17, 136, 264), (31, 64, 8), (33, 264, 129), (64, 512, 384), (127, 63, 255), (128, 128, 256), (129, 1001, 520),
    (200, 72, 3000), (256, 256, 512), (300, 1032, 777), (513, 264, 1032), (1000, 200, 100), (2049, 136, 72),
]


@pytest.mark.parametrize("n,k,m", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_linear(any_path, block, n, k, m, dtype):
    i = SHAPES.index((n, k, m))
    g = gen_of(100 + i)
    act = R.ACTS[i % 5]
    x, w = rnd(g, n, k), rnd(g, m, k, scale=k ** -0.5)
    sx = sw = None
    scale = 1.0
    if dtype == "e4m3":
        (x, sx), (w, sw) = codes(x), codes(w)
        scale = float(sx.double() * sw.double())
    unit = 16 if dtype == "e4m3" else 8
    bias = rnd(g, m) if i % 3 else None
    res = rnd(g, n, m) if i % 2 else None
    want = R.linear(d(x), d(w), d(bias), act, d(res), scale)
    y, z = Out(n, m), Out(n, m, extra=2)
    t.tpo_linear(block, pitched(x, unit, i % 3), pitched(w, unit, i % 2), y.t, bias=bias, act=ACT[act],
                 residual=None if res is None else pitched(res, 8, 1), z=z.t if i % 2 else None, scale_inv_x=sx,
                 scale_inv_w=sw)
    synced(block)
    R.check("y", y.get(), want["y"])
    if i % 2:
        R.check("z", z.get(), want["z"])


LARGE = [(1500, 1200, 3000), (4100, 520, 2104), (300, 4104, 1000), (2504, 264, 5000), (6000, 256, 264),
         (150, 264, 9000), (1030, 2056, 392)]


@pytest.mark.parametrize("n,k,m", LARGE)
def test_many_tiles(block, n, k, m):
    """Several rounds of tiles, long and short contractions, as the rule runs them."""
    g = gen_of(700 + LARGE.index((n, k, m)))
    x, w, w2 = rnd(g, n, k), rnd(g, m, k, scale=k ** -0.5), rnd(g, m, k, scale=k ** -0.5)
    bias, res, dy, z, u = rnd(g, m), rnd(g, n, m), rnd(g, n, m), rnd(g, n, m), rnd(g, n, m)
    y, zo, h = Out(n, m), Out(n, m), Out(n, m)
    dx, dw, gx, gg, gu = Out(n, k), Out(m, k), Out(n, k), Out(m, k), Out(m, k)
    db = torch.empty_like(bias)
    t.tpo_linear(block, x, w, y.t, bias=bias, act=ACT["gelu_tanh"], residual=res, z=zo.t)
    t.tpo_gated(block, x, w, w2, h.t, act=ACT["silu"])
    t.tpo_linear_bwd(block, dy, x, w, dx=dx.t, dw=dw.t, db=db, act=ACT["gelu"], z=z)
    t.tpo_gated_bwd(block, dy, z, u, x, w, w2, dx=gx.t, dwg=gg.t, dwu=gu.t)
    synced(block)
    want = R.linear(d(x), d(w), d(bias), "gelu_tanh", d(res))
    R.check("y", y.get(), want["y"])
    R.check("z", zo.get(), want["z"])
    R.check("h", h.get(), R.gated(d(x), d(w), d(w2), "silu")["h"])
    want = R.linear_bwd(d(dy), d(x), d(w), d(z), "gelu")
    for name, o in (("dx", dx.get()), ("dw", dw.get()), ("db", db)):
        R.check(name, o, want[name])
    want = R.gated_bwd(d(dy), d(z), d(u), d(x), d(w), d(w2))
    for name, o in (("dx", gx), ("dwg", gg), ("dwu", gu)):
        R.check(name, o.get(), want[name])


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n", [1, 70, 600])
def test_linear_every_epilogue(any_path, block, act, n):
    g = gen_of(n)
    k, m = 192, 328
    x, w, bias, res = rnd(g, n, k), rnd(g, m, k, scale=3 * k ** -0.5), rnd(g, m), rnd(g, n, m)
    for has_b in (0, 1):
        for has_r in (0, 1):
            for has_z in (0, 1):
                want = R.linear(d(x), d(w), d(bias) if has_b else None, act, d(res) if has_r else None)
                y, z = Out(n, m), Out(n, m)
                t.tpo_linear(block, x, w, y.t, bias=bias if has_b else None, act=ACT[act],
                             residual=res if has_r else None, z=z.t if has_z else None)
                synced(block)
                R.check("y", y.get(), want["y"])
                if has_z:
                    R.check("z", z.get(), want["z"])


@pytest.mark.parametrize("n", [1, 40, 700])
def test_linear_residual_in_place(any_path, block, n):
    g = gen_of(n)
    x, w, res = rnd(g, n, 256), rnd(g, 520, 256, scale=0.1), rnd(g, n, 520)
    want = R.linear(d(x), d(w), residual=d(res))
    t.tpo_linear(block, x, w, res, residual=res)
    synced(block)
    R.check("y", res, want["y"])


@pytest.mark.parametrize("n", [3, 300])
def test_not_finite_values_stay_in_their_row(any_path, block, n):
    g = gen_of(9)
    x, w = rnd(g, n, 264), rnd(g, 136, 264, scale=0.1)
    x[1, 5] = float("nan")
    x[2, 263] = float("inf")
    for act in R.ACTS:
        y, h = Out(n, 136), Out(n, 136)
        t.tpo_linear(block, x, w, y.t, act=ACT[act])
        t.tpo_gated(block, x, w, w.flip(0).contiguous(), h.t, act=ACT[act])
        synced(block)
        y, h = y.get().double(), h.get().double()
        xd, wd = d(x), d(w)
        keep = [r for r in range(n) if r not in (1, 2)]
        assert torch.isnan(y[1]).all() and torch.isnan(h[1]).all()
        assert torch.isfinite(y[keep]).all() and torch.isfinite(h[keep]).all()
        zinf = xd[2] @ wd.T
        want = R.act(zinf, act)
        assert (torch.isnan(y[2]) == torch.isnan(want)).all(), act
        ok = ~torch.isnan(want)
        assert (y[2][ok] == want.to(BF16).double()[ok]).all(), act


def test_large_values_of_the_activations(any_path, block):
    """Pre-activations far outside the functions' curved part, both signs."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 9.0, -9.0, 30.0, -30.0, 89.0, -89.0, 200.0, -200.0, 3e4, -3e4,
                      1e30, -1e30], device="cuda").to(BF16)
    n = z.numel()
    x = torch.zeros(n, 8, dtype=BF16, device="cuda")
    x[:, 0] = z
    w = torch.zeros(8, 8, dtype=BF16, device="cuda")
    w[:, 0] = 1
    dy = torch.ones(n, 8, dtype=BF16, device="cuda")
    for act in R.ACTS[1:]:
        want = R.linear(d(x), d(w), act_name=act)
        y = Out(n, 8)
        t.tpo_linear(block, x, w, y.t, act=ACT[act])
        synced(block)
        R.check(act, y.get(), want["y"])
        zz = z[:, None].expand(n, 8).contiguous()
        # dx's first column sums eight copies of act'(z)
        dx = Out(n, 8)
        t.tpo_linear_bwd(block, dy, x, w, dx=dx.t, act=ACT[act], z=zz)
        synced(block)
        R.check(act + "'", dx.get(), R.linear_bwd(d(dy), d(x), d(w), d(zz), act)["dx"])


@pytest.mark.parametrize("n,k,m", SHAPES)
def test_linear_bwd(any_path, block, n, k, m):
    i = SHAPES.index((n, k, m))
    g = gen_of(200 + i)
    act = R.ACTS[(i + 1) % 5]
    x, w, dy = rnd(g, n, k), rnd(g, m, k, scale=m ** -0.5), rnd(g, n, m)
    z = None if act == "none" else rnd(g, n, m, scale=1.5)
    want = R.linear_bwd(d(dy), d(x), d(w), d(z), act)
    dx, dw, db = Out(n, k), Out(m, k), torch.full((m,), float("nan"), dtype=BF16, device="cuda")
    t.tpo_linear_bwd(block, pitched(dy, 8, i % 2), pitched(x, 8, i % 3), pitched(w, 8, 1), dx=dx.t, dw=dw.t, db=db,
                     act=ACT[act], z=None if z is None else pitched(z, 8, 1))
    synced(block)
    R.check("dx", dx.get(), want["dx"])
    R.check("dw", dw.get(), want["dw"])
    R.check("db", db, want["db"])


@pytest.mark.parametrize("which", ["dx", "dw", "db", "dx dw", "dx db", "dw db", ""])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_bwd_parts(block, which, act):
    g = gen_of(7)
    n, k, m = 70, 136, 200
    x, w, dy = rnd(g, n, k), rnd(g, m, k), rnd(g, n, m)
    z = None if act == "none" else rnd(g, n, m)
    want = R.linear_bwd(d(dy), d(x), d(w), d(z), act)
    out = dict(dx=Out(n, k), dw=Out(m, k))
    db = torch.full((m,), float("nan"), dtype=BF16, device="cuda")
    parts = which.split()
    t.tpo_linear_bwd(block, dy, x if "dw" in parts else None, w if "dx" in parts else None,
                     dx=out["dx"].t if "dx" in parts else None, dw=out["dw"].t if "dw" in parts else None,
                     db=db if "db" in parts else None, act=ACT[act], z=z)
    synced(block)
    for p in parts:
        R.check(p, db if p == "db" else out[p].get(), want[p])


# ------------------------------------------------------------------ gated

@pytest.mark.parametrize("n,k,m", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_gated(any_path, block, n, k, m, dtype):
    i = SHAPES.index((n, k, m))
    gen = gen_of(300 + i)
    act = R.ACTS[(i + 4) % 5]
    x, wg, wu = rnd(gen, n, k), rnd(gen, m, k, scale=2 * k ** -0.5), rnd(gen, m, k, scale=k ** -0.5)
    sx = sg = su = None
    fg = fu = 1.0
    if dtype == "e4m3":
        (x, sx), (wg, sg), (wu, su) = codes(x), codes(wg), codes(wu)
        fg, fu = float(sx.double() * sg.double()), float(sx.double() * su.double())
    unit = 16 if dtype == "e4m3" else 8
    want = R.gated(d(x), d(wg), d(wu), act, fg, fu)
    h, go, uo = Out(n, m), Out(n, m, extra=2), Out(n, m, extra=3)
    save = i % 2 == 0
    t.tpo_gated(block, pitched(x, unit, i % 2), pitched(wg, unit, 1), pitched(wu, unit), h.t, act=ACT[act],
                g=go.t if save else None, u=uo.t if save else None, scale_inv_x=sx, scale_inv_wg=sg, scale_inv_wu=su)
    synced(block)
    R.check("h", h.get(), want["h"])
    if save:
        R.check("g", go.get(), want["g"])
        R.check("u", uo.get(), want["u"])


@pytest.mark.parametrize("n,k,m", SHAPES)
def test_gated_bwd(any_path, block, n, k, m):
    i = SHAPES.index((n, k, m))
    gen = gen_of(400 + i)
    act = R.ACTS[(i + 2) % 5]
    x, wg, wu, dh = rnd(gen, n, k), rnd(gen, m, k, scale=m ** -0.5), rnd(gen, m, k, scale=m ** -0.5), rnd(gen, n, m)
    g, u = rnd(gen, n, m, scale=1.5), rnd(gen, n, m)
    want = R.gated_bwd(d(dh), d(g), d(u), d(x), d(wg), d(wu), act)
    dx, dwg, dwu = Out(n, k), Out(m, k), Out(m, k, extra=2)
    t.tpo_gated_bwd(block, pitched(dh, 8, i % 2), pitched(g, 8, 1), pitched(u, 8), pitched(x, 8, i % 3), pitched(wg, 8),
                    pitched(wu, 8, 1), dx=dx.t, dwg=dwg.t, dwu=dwu.t, act=ACT[act])
    synced(block)
    R.check("dx", dx.get(), want["dx"])
    R.check("dwg", dwg.get(), want["dwg"])
    R.check("dwu", dwu.get(), want["dwu"])


@pytest.mark.parametrize("which", ["dx", "dw", ""])
def test_gated_bwd_parts(block, which):
    gen = gen_of(8)
    n, k, m = 70, 136, 200
    x, wg, wu, dh, g, u = (rnd(gen, *s) for s in ((n, k), (m, k), (m, k), (n, m), (n, m), (n, m)))
    want = R.gated_bwd(d(dh), d(g), d(u), d(x), d(wg), d(wu))
    dx, dwg, dwu = Out(n, k), Out(m, k), Out(m, k)
    t.tpo_gated_bwd(block, dh, g, u, x, wg, wu, dx=dx.t if which == "dx" else None,
                    dwg=dwg.t if which == "dw" else None, dwu=dwu.t if which == "dw" else None)
    synced(block)
    if which == "dx":
        R.check("dx", dx.get(), want["dx"])
    if which == "dw":
        R.check("dwg", dwg.get(), want["dwg"])
        R.check("dwu", dwu.get(), want["dwu"])


@pytest.mark.parametrize("act", R.ACTS)
def test_gradients_against_differences(block, act):
    """<gradient, direction> from the kernels against the central difference of the definition in 64 bits."""
    gen = gen_of(11)
    n, k, m = 24, 40, 56
    x, w, w2, dy = rnd(gen, n, k), rnd(gen, m, k, scale=0.2), rnd(gen, m, k, scale=0.2), rnd(gen, n, m)
    lin = R.linear(d(x), d(w), act_name=act)
    z = None if act == "none" else lin["z"][0].to(BF16)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    t.tpo_linear_bwd(block, dy, x, w, dx=dx, dw=dw, act=ACT[act], z=z)
    gat = R.gated(d(x), d(w), d(w2), act)
    gx, gg, gu = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    t.tpo_gated_bwd(block, dy, gat["g"][0].to(BF16), gat["u"][0].to(BF16), x, w, w2, dx=gx, dwg=gg, dwu=gu,
                    act=ACT[act])
    synced(block)
    f1 = lambda x, w: (R.linear(x, w, act_name=act)["y"][0] * d(dy)).sum()  # noqa: E731
    f2 = lambda x, wg, wu: (R.gated(x, wg, wu, act)["h"][0] * d(dy)).sum()  # noqa: E731
    for f, ins, grads in ((f1, dict(x=x, w=w), dict(x=dx, w=dw)),
                          (f2, dict(x=x, wg=w, wu=w2), dict(x=gx, wg=gg, wu=gu))):
        for name in ins:
            v = rnd(gen, *ins[name].shape, dtype=torch.float64)
            hh = 1e-5
            up, dn = {q: d(s) for q, s in ins.items()}, {q: d(s) for q, s in ins.items()}
            up[name], dn[name] = up[name] + hh * v, dn[name] - hh * v
            diff = float(f(**up) - f(**dn)) / (2 * hh)
            got = d(grads[name])
            # each gradient element is off by a few roundings to bf16 of terms its own size; relu's kink may
            # fall between z and its bf16 value, which the saved z decides
            tol = 8 * R.U16 * float((got.abs() * v.abs()).square().sum().sqrt()) * 4 + 1e-3 * abs(diff)
            assert abs(float((got * v).sum()) - diff) <= tol, (act, name)


# ------------------------------------------------------------------ layer norm

NORMS = [(1, 1), (2, 2), (3, 7), (1, 64), (5, 100), (4, 255), (7, 256), (129, 1000), (3, 1024), (33, 1029), (2, 2048),
         (160, 4096), (6, 5003), (3, 8192), (5, 8200), (2, 16384), (3, 20001), (2, 40000), (2000, 8), (1500, 72),
         (4200, 520), (4000, 1003), (1000, 5003), (900, 7001), (700, 8192), (3000, 2048), (500, 12288), (9000, 136)]


@pytest.mark.parametrize("n,k", NORMS)
@pytest.mark.parametrize("dt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm(block, n, k, dt, wt):
    i = NORMS.index((n, k))
    g = gen_of(500 + i)
    x = rnd(g, n, k, dtype=dt, scale=3) + (5.0 if i % 2 else 0.0)
    gamma = rnd(g, k, dtype=wt) if i % 4 != 3 else None
    beta = rnd(g, k, dtype=wt) if i % 3 != 2 else None
    # odd pitches and bases on every other case
    odd = i % 2 == 0
    xin = pitched(x, 1, 3) if odd else x
    y = Out(n, k, dt, unit=1 if odd else 8, extra=5 if odd else 1)
    want = R.layer_norm(d(x), d(gamma), d(beta), 1e-5)
    mean, rstd = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    t.tpo_layer_norm(block, xin, gamma, beta, y.t, mean=mean, rstd=rstd)
    synced(block)
    R.check("y", y.get(), want["y"])
    R.check("mean", mean, want["mean"])
    R.check("rstd", rstd, want["rstd"])


@pytest.mark.parametrize("n,k", NORMS)
@pytest.mark.parametrize("dt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm_bwd(block, n, k, dt, wt):
    i = NORMS.index((n, k))
    g = gen_of(600 + i)
    x, dy = rnd(g, n, k, dtype=dt, scale=3) + (5.0 if i % 2 else 0.0), rnd(g, n, k, dtype=dt)
    gamma = rnd(g, k, dtype=wt) if i % 4 != 3 else None
    dres = rnd(g, n, k, dtype=dt) if i % 3 else None
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    odd = i % 2 == 0
    dx = Out(n, k, dt, unit=1 if odd else 8, extra=5 if odd else 1)
    dg, db = (torch.full((k,), float("nan"), dtype=wt, device="cuda") for _ in range(2))
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    t.tpo_layer_norm_bwd(block, pitched(dy, 1, 1) if odd else dy, pitched(x, 1, 2) if odd else x, gamma, mean, rstd,
                         dx.t, dgamma=dg, dbeta=db, dres=dres)
    synced(block)
    R.check("dx", dx.get(), want["dx"])
    R.check("dgamma", dg, want["dgamma"])
    R.check("dbeta", db, want["dbeta"])


# Aligned rows that give a thread each number of vectors, exactly or with some left over, in many rows and in few.
WIDTHS = [(1700, 640), (1700, 768), (900, 1280), (900, 1248), (1700, 1024), (700, 2560), (700, 2504), (300, 5120),
          (250, 6144), (220, 8448), (130, 9000), (120, 12288), (110, 16384), (105, 20480), (16400, 264), (16400, 512)]


@pytest.mark.parametrize("n,k", WIDTHS)
@pytest.mark.parametrize("dt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_layer_norm_widths(block, n, k, dt, wt):
    i = WIDTHS.index((n, k))
    g = gen_of(700 + i)
    x, dy = rnd(g, n, k, dtype=dt, scale=3) + 2.0, rnd(g, n, k, dtype=dt)
    gamma = rnd(g, k, dtype=wt) if i % 4 != 3 else None
    beta = rnd(g, k, dtype=wt) if i % 3 != 2 else None
    dres = rnd(g, n, k, dtype=dt) if i % 2 else None
    want = R.layer_norm(d(x), d(gamma), d(beta), 1e-5)
    y = Out(n, k, dt, unit=8, extra=1)
    mean, rstd = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    t.tpo_layer_norm(block, x, gamma, beta, y.t, mean=mean, rstd=rstd)
    synced(block)
    for name, v in (("y", y.get()), ("mean", mean), ("rstd", rstd)):
        R.check(name, v, want[name])
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    dx = Out(n, k, dt, unit=8, extra=1)
    dg, db = (torch.full((k,), float("nan"), dtype=wt, device="cuda") for _ in range(2))
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dx.t, dgamma=dg, dbeta=db, dres=dres)
    synced(block)
    for name, v in (("dx", dx.get()), ("dgamma", dg), ("dbeta", db)):
        R.check(name, v, want[name])


# Rows shorter than a warp, many and few of them.
@pytest.mark.parametrize("n,k", [(22001, 64), (100000, 8), (22000, 40), (11003, 128), (6000, 120), (300, 64), (1, 8)])
@pytest.mark.parametrize("dt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("parts", ["all", "plain", "weights"])
def test_layer_norm_bwd_short_rows(block, n, k, dt, wt, parts):
    g = gen_of(n + k)
    x, dy = rnd(g, n, k, dtype=dt, scale=2) + 1.0, rnd(g, n, k, dtype=dt)
    gamma = rnd(g, k, dtype=wt) if parts != "plain" else None
    dres = rnd(g, n, k, dtype=dt) if parts == "all" else None
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    dx = Out(n, k, dt, unit=8, extra=1)
    dg, db = (torch.full((k,), float("nan"), dtype=wt, device="cuda") for _ in range(2))
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, None if parts == "weights" else dx.t,
                         dgamma=None if parts == "plain" else dg, dbeta=None if parts == "plain" else db, dres=dres)
    synced(block)
    if parts != "weights":
        R.check("dx", dx.get(), want["dx"])
    if parts != "plain":
        R.check("dgamma", dg, want["dgamma"])
        R.check("dbeta", db, want["dbeta"])


@pytest.mark.parametrize("n,k", [(1200, 1003), (400, 5003), (1100, 4096), (2000, 24)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_layer_norm_many_rows_in_place(block, n, k, dt):
    g = gen_of(n)
    x, dy, gamma, beta = rnd(g, n, k, dtype=dt), rnd(g, n, k, dtype=dt), rnd(g, k, dtype=dt), rnd(g, k, dtype=dt)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    y = x.clone()
    t.tpo_layer_norm(block, y, gamma, beta, y, mean=mean, rstd=rstd)
    synced(block)
    R.check("y", y, R.layer_norm(d(x), d(gamma), d(beta), 1e-5)["y"])
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd))
    dg, db = torch.empty_like(gamma), torch.empty_like(beta)
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dy, dgamma=dg, dbeta=db)
    synced(block)
    for name, v in (("dx", dy), ("dgamma", dg), ("dbeta", db)):
        R.check(name, v, want[name])


@pytest.mark.parametrize("which", ["dx", "dgamma", "dbeta", "dx dgamma", "dgamma dbeta", ""])
def test_layer_norm_bwd_parts(block, which):
    g = gen_of(12)
    n, k = 70, 1000
    x, dy, gamma = rnd(g, n, k), rnd(g, n, k), rnd(g, k)
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd))
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    parts = which.split()
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dx if "dx" in parts else None,
                         dgamma=dg if "dgamma" in parts else None, dbeta=db if "dbeta" in parts else None)
    synced(block)
    for name, v in (("dx", dx), ("dgamma", dg), ("dbeta", db)):
        if name in parts:
            R.check(name, v, want[name])


@pytest.mark.parametrize("k", [96, 4096, 5003, 40000])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_layer_norm_in_place_and_special_rows(block, k, dt):
    g = gen_of(k)
    x = rnd(g, 8, k, dtype=dt)
    x[1] = 2.5           # no variance: rstd is 1 / sqrt(eps)
    x[2, k // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] = 0
    x[5] += 1000.0       # a mean far above the spread
    gamma, beta = rnd(g, k, dtype=F32), rnd(g, k, dtype=F32)
    keep = [0, 1, 4, 5, 6, 7]
    want = R.layer_norm(d(x[keep]), d(gamma), d(beta), 1e-5)
    mean, rstd = torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    t.tpo_layer_norm(block, x, gamma, beta, x, mean=mean, rstd=rstd)
    synced(block)
    R.check("y", x[keep], want["y"])
    R.check("rstd", rstd[keep], want["rstd"])
    assert torch.isnan(x[2]).all() and torch.isnan(x[3]).all()


@pytest.mark.parametrize("onto", ["dy", "dres"])
@pytest.mark.parametrize("n,k", [(40, 520), (700, 4096), (3, 40000)])
def test_layer_norm_bwd_in_place(block, onto, n, k):
    g = gen_of(13)
    x, dy, gamma, dres = rnd(g, n, k), rnd(g, n, k), rnd(g, k), rnd(g, n, k)
    f = R.layer_norm(d(x), d(gamma), None, 1e-5)
    mean, rstd = f["mean"][0].float(), f["rstd"][0].float()
    want = R.layer_norm_bwd(d(dy), d(x), d(gamma), d(mean), d(rstd), d(dres))
    dg, db = torch.empty_like(gamma), torch.empty_like(gamma)
    dx = dict(dy=dy, dres=dres)[onto]
    t.tpo_layer_norm_bwd(block, dy, x, gamma, mean, rstd, dx, dgamma=dg, dbeta=db, dres=dres)
    synced(block)
    R.check("dx", dx, want["dx"])
    R.check("dgamma", dg, want["dgamma"])
    R.check("dbeta", db, want["dbeta"])


# ------------------------------------------------------------------ the calls

def test_empty_batch(block):
    g = gen_of(14)
    e = lambda c: torch.empty(0, c, dtype=BF16, device="cuda")  # noqa: E731
    w, w2, gamma = rnd(g, 24, 16), rnd(g, 24, 16), rnd(g, 16)
    t.tpo_linear(block, e(16), w, e(24), bias=rnd(g, 24), residual=e(24), z=e(24), act=ACT["gelu"])
    t.tpo_gated(block, e(16), w, w2, e(24), g=e(24), u=e(24))
    v = torch.empty(0, device="cuda")
    t.tpo_layer_norm(block, e(16), gamma, gamma, e(16), mean=v, rstd=v)
    dw, dw2, dw3 = Out(24, 16), Out(24, 16), Out(24, 16)
    db, dg, dbt = (torch.full((c,), float("nan"), dtype=BF16, device="cuda") for c in (24, 16, 16))
    t.tpo_linear_bwd(block, e(24), e(16), w, dx=e(16), dw=dw.t, db=db, act=ACT["relu"], z=e(24))
    t.tpo_gated_bwd(block, e(24), e(24), e(24), e(16), w, w2, dx=e(16), dwg=dw2.t, dwu=dw3.t)
    t.tpo_layer_norm_bwd(block, e(16), e(16), gamma, v, v, e(16), dgamma=dg, dbeta=dbt)
    synced(block)
    for o in (dw.get(), dw2.get(), dw3.get(), db, dg, dbt):
        assert (o == 0).all()


def _all_calls(block, s):
    t.tpo_layer_norm(block, s["x"], s["gamma"], s["beta"], s["y"], mean=s["mean"], rstd=s["rstd"])
    t.tpo_gated(block, s["y"], s["wg"], s["wu"], s["h"], g=s["g"], u=s["u"])
    t.tpo_linear(block, s["h"], s["wd"], s["o"], residual=s["x"], bias=s["b"])
    t.tpo_linear_bwd(block, s["do"], s["h"], s["wd"], dx=s["dh"], dw=s["dwd"], db=s["dbias"])
    t.tpo_gated_bwd(block, s["dh"], s["g"], s["u"], s["y"], s["wg"], s["wu"], dx=s["dy"], dwg=s["dwg"], dwu=s["dwu"])
    t.tpo_layer_norm_bwd(block, s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], dgamma=s["dga"],
                         dbeta=s["dbe"], dres=s["do"])
    return [s[q] for q in ("y", "h", "o", "dh", "dwd", "dbias", "dy", "dwg", "dwu", "dx", "dga", "dbe")]


def _layer(n, k, m, seed):
    g = gen_of(seed)
    e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    return dict(x=rnd(g, n, k), gamma=rnd(g, k), beta=rnd(g, k), wg=rnd(g, m, k, scale=k ** -0.5),
                wu=rnd(g, m, k, scale=k ** -0.5), wd=rnd(g, k, m, scale=m ** -0.5), b=rnd(g, k), do=rnd(g, n, k),
                y=e(n, k), mean=e(n, dtype=F32), rstd=e(n, dtype=F32), g=e(n, m), u=e(n, m), h=e(n, m), o=e(n, k),
                dh=e(n, m), dwd=e(k, m), dbias=e(k), dy=e(n, k), dwg=e(m, k), dwu=e(m, k), dx=e(n, k), dga=e(k),
                dbe=e(k))


@pytest.mark.parametrize("n,k,m", [(1, 256, 384), (50, 520, 264), (700, 512, 1024)])
def test_layer_step_matches_its_steps(any_path, block, n, k, m):
    """The whole feed-forward sublayer, forward and backward, each step against its definition on that step's inputs."""
    s = _layer(n, k, m, n)
    _all_calls(block, s)
    synced(block)
    q = {a: d(v) for a, v in s.items()}
    R.check("y", s["y"], R.layer_norm(q["x"], q["gamma"], q["beta"], 1e-5)["y"])
    R.check("h", s["h"], R.gated(q["y"], q["wg"], q["wu"])["h"])
    R.check("o", s["o"], R.linear(q["h"], q["wd"], q["b"], residual=q["x"])["y"])
    w = R.linear_bwd(q["do"], q["h"], q["wd"])
    R.check("dh", s["dh"], w["dx"])
    R.check("dwd", s["dwd"], w["dw"])
    w = R.gated_bwd(q["dh"], q["g"], q["u"], q["y"], q["wg"], q["wu"])
    R.check("dy", s["dy"], w["dx"])
    R.check("dwg", s["dwg"], w["dwg"])
    w = R.layer_norm_bwd(q["dy"], q["x"], q["gamma"], q["mean"], q["rstd"], q["do"])
    R.check("dx", s["dx"], w["dx"])
    R.check("dga", s["dga"], w["dgamma"])


@pytest.mark.parametrize("n,k,m", [(1, 256, 384), (33, 520, 264), (1100, 512, 1032)])
def test_repeats_streams_and_graphs_give_the_same_bits(any_path, block, n, k, m):
    s = _layer(n, k, m, 5)
    first = [v.clone() for v in _all_calls(block, s)]
    for _ in range(3):
        again = _all_calls(block, s)
    synced(block)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    for v in again:
        v.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _all_calls(block, s)
        assert t.tpo_block_sync_status(block) == 0
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    for v in got:
        v.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_calls(block, s)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    synced(block)
    assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_options_round_trip(block):
    for key, value in (("path", 2), ("path", 0), ("split", 8), ("split", 0)):
        t.tpo_block_set_opt(block, key, value)
        assert t.tpo_block_get_opt(block, key) == value
    with pytest.raises(t.TpoError, match="path"):
        t.tpo_block_set_opt(block, "path", 3)


def test_workspace_and_device_checks():
    g = gen_of(15)
    b = t.tpo_block_create(0)
    try:
        x, w, z = rnd(g, 16, 16), rnd(g, 16, 16), rnd(g, 16, 16)
        with pytest.raises(t.TpoError, match="workspace"):
            t.tpo_linear_bwd(b, x, x, w, dx=torch.empty_like(x), act=ACT["gelu"], z=z)
        with pytest.raises(t.TpoError, match="workspace"):
            t.tpo_gated_bwd(b, x, x, x, x, w, w, dx=torch.empty_like(x))
        # no activation needs no workspace
        dx = torch.empty_like(x)
        t.tpo_linear_bwd(b, x, x, w, dx=dx)
        assert t.tpo_block_sync_status(b) == 0
        R.check("dx", dx, R.linear_bwd(d(x), d(x), d(w))["dx"])
        with pytest.raises(t.TpoError, match="shape"):
            t.tpo_linear(b, x, w[:, :8], dx)
        with pytest.raises(t.TpoError, match="type"):
            t.tpo_linear(b, x, w.float(), dx)
        with pytest.raises(t.TpoError, match="unit stride"):
            t.tpo_linear(b, x, w.T, dx)
        with pytest.raises(t.TpoError, match="pitch"):
            t.tpo_linear(b, rnd(g, 4, 9), rnd(g, 16, 9), torch.empty(4, 16, dtype=BF16, device="cuda"))
    finally:
        t.tpo_block_destroy(b)


def test_offsets_past_32_bits(any_path, block):
    """Matrices whose last elements lie past 2^31 elements from their first."""
    pitch = 1 << 24
    big = torch.zeros(144, pitch, dtype=BF16, device="cuda")  # 2.4e9 elements, 4.8 GB
    g = gen_of(16)
    n, k, m = 144, 264, 136
    x = big[:, :k]
    x.copy_(rnd(g, n, k))
    w = rnd(g, m, k, scale=0.1)
    y = torch.empty(n, m, dtype=BF16, device="cuda")
    t.tpo_linear(block, x, w, y)
    far = big[:, 512:512 + k]
    t.tpo_layer_norm(block, x, None, None, far)
    back, dw = big[:, 1024:1024 + k], torch.empty_like(w)
    t.tpo_linear_bwd(block, y, x, w, dx=back, dw=dw)
    synced(block)
    R.check("y", y, R.linear(d(x), d(w))["y"])
    R.check("norm", far, R.layer_norm(d(x), None, None, 1e-5)["y"])
    want = R.linear_bwd(d(y), d(x), d(w))
    R.check("dx", back, want["dx"])
    R.check("dw", dw, want["dw"])


# the stages' roundings to bf16 (norm, g, u, h, dh, dg, du, dnorm) add up to a few 2^-8 of each result's size
@pytest.mark.parametrize("args", ["--tokens 300 --hidden 256 --ffn 384 --train", "--tokens 1 --hidden 512 --ffn 768",
                                  "--tokens 512 --hidden 256 --ffn 512 --tp 2"])
def test_example_layer(args):
    from tensor_comm_gemm_gb300 import ffn_layer
    errors = ffn_layer.main(args.split() + ["--check", "--calls", "2"])
    assert errors and all(e < 4 * R.U16 for e in errors.values()), errors
