"""The block operators without a GPU: workspace sizes, refusals (raised before
the handle or CUDA is touched) and the references' own gradients against
differences."""

import ctypes

import pytest
import torch

import block_ref as R
from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t

INVALID, UNSUPPORTED = t.TPO_ERR_INVALID_ARG, t.TPO_ERR_UNSUPPORTED
P = 0x10000  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


def test_workspace_sizes(lib):
    for op in (t.TPO_OP_LAYER_NORM, t.TPO_OP_LINEAR, t.TPO_OP_GATED):
        assert t.tpo_block_workspace(op, 4096, 4096, 4096) == 0
    for n, k, m in ((0, 1, 1), (1, 1, 1), (777, 1000, 333), (1 << 20, 1 << 14, 1 << 14)):
        # at least the gradient of the pre-activation, in bf16
        assert t.tpo_block_workspace(t.TPO_OP_LINEAR_BWD, n, k, m) >= 2 * n * m
        assert t.tpo_block_workspace(t.TPO_OP_GATED_BWD, n, k, m) >= 4 * n * m
        assert t.tpo_block_workspace(t.TPO_OP_LAYER_NORM_BWD, n, k) >= 0


@pytest.mark.parametrize("op,n,k,m", [(6, 1, 1, 1), (-1, 1, 1, 1), (2, -1, 8, 8), (2, 1, 0, 8), (2, 1, 8, 0),
                                      (2, (1 << 30) + 1, 8, 8), (0, 1, 0, 1)])
def test_workspace_refuses(lib, op, n, k, m):
    assert lib.tpo_block_workspace(op, n, k, m) == -1
    assert t.tpo_last_error()


def test_create_and_null_handles(lib):
    assert not lib.tpo_block_create(-1)
    assert "workspace" in t.tpo_last_error()
    assert lib.tpo_block_destroy(None) == 0
    assert lib.tpo_block_sync_status(None, None) == INVALID


def test_options_refuse(lib):
    for key, value, word in ((b"path", 3, "path"), (b"path", -1, "path"), (b"split", 9, "split"), (b"other", 0, "other"),
                             (b"path", 1, "handle")):
        assert lib.tpo_block_set_opt(None, key, value) == INVALID
        assert word in t.tpo_last_error()
    assert lib.tpo_block_set_opt(None, None, 0) == INVALID
    assert lib.tpo_block_get_opt(None, b"path", None) == INVALID
    assert lib.tpo_block_get_opt(None, b"path", ctypes.byref(ctypes.c_int64())) == INVALID


def linear(lib, n=4, k=16, m=8, dtype=0, x=P, ldx=16, w=P, ldw=16, bias=None, act=0, r=None, ldr=8, z=None, ldz=8,
           y=P, ldy=8, sx=None, sw=None):
    return lib.tpo_linear(None, n, k, m, dtype, x, ldx, w, ldw, bias, act, r, ldr, z, ldz, y, ldy, sx, sw, None)


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=-1), INVALID, "sizes"), (dict(k=0), INVALID, "sizes"), (dict(m=0), INVALID, "sizes"),
    (dict(m=(1 << 30) + 1), INVALID, "sizes"),
    (dict(act=5), INVALID, "act"), (dict(act=-1), INVALID, "act"),
    (dict(dtype=2), INVALID, "dtype"), (dict(dtype=7), INVALID, "dtype"),
    (dict(sx=P), INVALID, "scale"), (dict(dtype=1, sx=P), INVALID, "scale"),
    (dict(dtype=1, sx=P, sw=P + 1), INVALID, "scale"),
    (dict(x=None), INVALID, "x"), (dict(x=P + 2), INVALID, "x"), (dict(w=None), INVALID, "w"),
    (dict(w=P + 8), INVALID, "w"), (dict(y=None), INVALID, "y"), (dict(y=P + 4), INVALID, "y"),
    (dict(ldx=15), INVALID, "x"), (dict(ldx=18), UNSUPPORTED, "x"), (dict(ldw=8), INVALID, "w"),
    (dict(ldw=20), UNSUPPORTED, "w"), (dict(ldy=12), UNSUPPORTED, "y"), (dict(ldy=0), INVALID, "y"),
    (dict(dtype=1, ldx=24, sx=P, sw=P), UNSUPPORTED, "x"),
    (dict(r=P + 2), INVALID, "residual"), (dict(r=P, ldr=9), UNSUPPORTED, "residual"),
    (dict(z=P + 2), INVALID, "z"), (dict(z=P, ldz=7), INVALID, "z"), (dict(bias=P + 1), INVALID, "bias"),
    (dict(), INVALID, "handle"),
])
def test_linear_refuses(lib, kw, status, word):
    assert linear(lib, **kw) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=-1), INVALID, "sizes"), (dict(act=9), INVALID, "act"), (dict(act=1), INVALID, "z"),
    (dict(z=P), INVALID, "z"), (dict(dy=None), INVALID, "dy"), (dict(lddy=12), UNSUPPORTED, "dy"),
    (dict(dx=P + 2), INVALID, "dx"), (dict(w=None), INVALID, "w"), (dict(x=None), INVALID, "x"),
    (dict(dw=P, lddw=15), INVALID, "dw"), (dict(db=P + 1), INVALID, "db"), (dict(), INVALID, "handle"),
])
def test_linear_bwd_refuses(lib, kw, status, word):
    a = dict(n=4, k=16, m=8, act=0, dy=P, lddy=8, z=None, ldz=8, x=P, ldx=16, w=P, ldw=16, dx=P, lddx=16, dw=P,
             lddw=16, db=None)
    a.update(kw)
    assert lib.tpo_linear_bwd(None, *a.values(), None) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(k=0), INVALID, "sizes"), (dict(dtype=2), INVALID, "dtype"), (dict(act=7), INVALID, "act"),
    (dict(wg=None), INVALID, "wg"), (dict(wu=P + 2), INVALID, "wu"), (dict(ldwu=17), UNSUPPORTED, "wu"),
    (dict(h=None), INVALID, "h"), (dict(g=P), INVALID, "g and u"), (dict(u=P), INVALID, "g and u"),
    (dict(g=P, u=P, ldu=4), INVALID, "u"), (dict(swu=P), INVALID, "scale"),
    (dict(dtype=1, sx=P, swg=P), INVALID, "scale"), (dict(), INVALID, "handle"),
])
def test_gated_refuses(lib, kw, status, word):
    a = dict(n=4, k=16, m=8, dtype=0, x=P, ldx=16, wg=P, ldwg=16, wu=P, ldwu=16, act=4, g=None, ldg=8, u=None, ldu=8,
             h=P, ldh=8, sx=None, swg=None, swu=None)
    a.update(kw)
    assert lib.tpo_gated(None, *a.values(), None) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(m=0), INVALID, "sizes"), (dict(act=-2), INVALID, "act"), (dict(g=None), INVALID, "g"),
    (dict(u=P + 2), INVALID, "u"), (dict(lddh=9), UNSUPPORTED, "dh"), (dict(dwg=None), INVALID, "dwg"),
    (dict(dwu=None), INVALID, "dwg"), (dict(wu=None), INVALID, "wu"), (dict(x=None), INVALID, "x"),
    (dict(lddx=8), INVALID, "dx"), (dict(), INVALID, "handle"),
])
def test_gated_bwd_refuses(lib, kw, status, word):
    a = dict(n=4, k=16, m=8, act=4, dh=P, lddh=8, g=P, ldg=8, u=P, ldu=8, x=P, ldx=16, wg=P, ldwg=16, wu=P, ldwu=16,
             dx=P, lddx=16, dwg=P, lddwg=16, dwu=P, lddwu=16)
    a.update(kw)
    assert lib.tpo_gated_bwd(None, *a.values(), None) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), "sizes"), (dict(k=0), "sizes"), (dict(dtype=1), "types"), (dict(wdtype=3), "types"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(x=None), "x"), (dict(x=P + 1), "x"),
    (dict(dtype=2, x=P + 2), "x"), (dict(ldx=9), "x"), (dict(y=None), "y"), (dict(gamma=P + 1), "gamma"),
    (dict(wdtype=2, beta=P + 2), "beta"), (dict(mean=P + 2), "mean"), (dict(rstd=P + 1), "rstd"), (dict(), "handle"),
])
def test_layer_norm_refuses(lib, kw, word):
    a = dict(n=4, k=10, dtype=0, wdtype=0, x=P, ldx=10, gamma=P, beta=P, eps=1e-5, y=P, ldy=10, mean=None, rstd=None)
    a.update(kw)
    assert lib.tpo_layer_norm(None, *a.values(), None) == INVALID
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(n=1 << 31), "sizes"), (dict(dtype=1), "types"), (dict(dy=None), "dy"), (dict(lddy=3), "dy"),
    (dict(dres=P + 1), "dres"), (dict(dx=P + 1), "dx"), (dict(mean=None), "mean"), (dict(rstd=None), "rstd"),
    (dict(dgamma=P + 1), "dgamma"), (dict(mean=P + 2), "mean"), (dict(), "handle"),
])
def test_layer_norm_bwd_refuses(lib, kw, word):
    a = dict(n=4, k=10, dtype=0, wdtype=0, dy=P, lddy=10, x=P, ldx=10, gamma=P, mean=P, rstd=P, dres=None, lddres=10,
             dx=P, lddx=10, dgamma=P, dbeta=P)
    a.update(kw)
    assert lib.tpo_layer_norm_bwd(None, *a.values(), None) == INVALID
    assert word in t.tpo_last_error(), t.tpo_last_error()


def test_binding_refuses_host_tensors_and_types(lib):
    x, w, y = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 8)
    b16 = torch.bfloat16
    with pytest.raises(t.TpoError, match="CUDA"):
        t.tpo_linear(1, x.to(b16), w.to(b16), y.to(b16))
    with pytest.raises(t.TpoError, match="2-D"):
        t.tpo_linear(1, x[0], w, y)
    with pytest.raises(t.TpoError, match="type"):
        t.tpo_layer_norm(1, x.double(), None, None, x)


def _directional(f, grads, inputs, gen):
    """<grad, d> against the central difference of f along d, for a random direction d of each input."""
    for name, g in grads.items():
        d = torch.randn(inputs[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = dict(inputs), dict(inputs)
        up[name], down[name] = inputs[name] + h * d, inputs[name] - h * d
        diff = (f(**up) - f(**down)) / (2 * h)
        assert abs(float((g * d).sum() - diff)) <= 1e-6 * (1 + abs(float(diff))), name


@pytest.mark.parametrize("act", R.ACTS)
def test_reference_gradients_against_differences(act):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, dy, w2 = r(5, 7), r(6, 7), r(6), r(5, 6), r(6, 7)
    z = R.linear(x, w, b, act)["z"][0]
    g = R.linear_bwd(dy, x, w, None if act == "none" else z, act)
    _directional(lambda x, w, b: (R.linear(x, w, b, act)["y"][0] * dy).sum(),
                 dict(x=g["dx"][0], w=g["dw"][0], b=g["db"][0]), dict(x=x, w=w, b=b), gen)
    f = R.gated(x, w, w2, act)
    g = R.gated_bwd(dy, f["g"][0], f["u"][0], x, w, w2, act)
    _directional(lambda x, wg, wu: (R.gated(x, wg, wu, act)["h"][0] * dy).sum(),
                 dict(x=g["dx"][0], wg=g["dwg"][0], wu=g["dwu"][0]), dict(x=x, wg=w, wu=w2), gen)


def test_reference_norm_gradient_against_differences():
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, ga, be, dy = r(5, 11), r(11), r(11), r(5, 11)
    f = R.layer_norm(x, ga, be, 1e-3)
    g = R.layer_norm_bwd(dy, x, ga, f["mean"][0], f["rstd"][0])
    _directional(lambda x, ga, be: (R.layer_norm(x, ga, be, 1e-3)["y"][0] * dy).sum(),
                 dict(x=g["dx"][0], ga=g["dgamma"][0], be=g["dbeta"][0]), dict(x=x, ga=ga, be=be), gen)


def test_check_sees_a_planted_mistake():
    """The bound is tight enough to see one wrong term of a sum, and one column's bias left out."""
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16().double()  # noqa: E731
    x, w, b = r(8, 256), r(16, 256), r(16)
    want = R.linear(x, w, b, "silu")["y"]
    R.check("y", want[0].bfloat16(), want)
    short = R.linear(x[:, :-1], w[:, :-1], b, "silu")["y"][0].bfloat16()
    with pytest.raises(AssertionError):
        R.check("y", short, want)
    b2 = b.clone()
    b2[3] = 0
    with pytest.raises(AssertionError):
        R.check("y", R.linear(x, w, b2, "silu")["y"][0].bfloat16(), want)
