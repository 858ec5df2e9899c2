"""The attention sublayer's operators without a GPU: tables, workspace sizes,
refusals (raised before the handle or CUDA is touched) and the references' own
gradients against differences."""

import ctypes
import math

import pytest
import torch

import attn_ref as A
import block_ref as R
from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t

INVALID, UNSUPPORTED = t.TPO_ERR_INVALID_ARG, t.TPO_ERR_UNSUPPORTED
P = 0x10000  # an aligned address that no refused call may touch


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


# ------------------------------------------------------------------ tables

@pytest.mark.parametrize("rot,base,scaling,kw", [
    (128, 10000.0, "none", {}), (64, 500000.0, "linear", dict(factor=8.0)), (2, 10000.0, "none", {}),
    (20, 1e6, "parts", dict(factor=4.0, low=1.0, high=4.0, original=8192)),
    (128, 500000.0, "parts", dict(factor=8.0, low=1.0, high=4.0, original=8192)), (0, 10000.0, "none", {})])
def test_table_entries(lib, rot, base, scaling, kw):
    code = dict(none=t.TPO_ROTARY_UNSCALED, linear=t.TPO_ROTARY_LINEAR, parts=t.TPO_ROTARY_BY_PARTS)[scaling]
    table = t.tpo_rotary_table(rot, base, code, **kw)
    want = A.frequencies(rot, base, scaling, **kw) / (2 * math.pi)
    assert table.shape == want.shape
    for got, turns in zip(table.tolist(), want.tolist()):
        got = (got % 2 ** 64) / 2 ** 64
        assert abs(got - turns % 1.0) <= 4 * 2.0 ** -53 * turns + 2.0 ** -63


@pytest.mark.parametrize("kw,word", [
    (dict(rot=3), "rot"), (dict(rot=-2), "rot"), (dict(rot=1 << 20), "rot"), (dict(base=0.0), "base"),
    (dict(base=math.nan), "base"), (dict(base=math.inf), "base"), (dict(scaling=3), "scaling"),
    (dict(scaling=1, factor=0.0), "factor"), (dict(scaling=2, factor=math.inf), "factor"),
    (dict(scaling=2, low=4.0, high=4.0), "low"), (dict(scaling=2, original=0), "original"),
    (dict(table=None), "table")])
def test_table_refuses(lib, kw, word):
    a = dict(rot=8, base=1e4, scaling=0, factor=2.0, low=1.0, high=4.0, original=10,
             table=ctypes.addressof((ctypes.c_uint64 * 4)()))
    a.update(kw)
    assert lib.tpo_rotary_table(*a.values()) == INVALID
    assert word in t.tpo_last_error(), t.tpo_last_error()


# ------------------------------------------------------------------ refusals

def test_workspace(lib):
    for f in (t.tpo_attention_workspace, t.tpo_attention_bwd_workspace):
        assert f(0, 0, 1, 1, 8) >= 0
        assert f(1 << 20, 1 << 20, 128, 1, 128) >= f(1, 1, 1, 1, 8)
        for bad in ((-1, 0, 1, 1, 8), (1, -1, 1, 1, 8), (1, 1, 3, 2, 8), (1, 1, 0, 1, 8), (1, 1, 1, 0, 8),
                    (1, 1, 1, 1, 0), (1, 1, 1, 1, 136), (1, 1, 1, 1, 12), (1, 1, 129, 1, 64)):
            with pytest.raises(t.TpoError):
                f(*bad)


SHAPE = dict(batch=2, n=4, nk=6, heads=4, kv_heads=2, dim=16, q_start=P, k_start=P, k_len=P, causal=1, scale=0.25)
ALONE = dict(batch=1, q_start=None, k_start=None, k_len=None)
COMMON = [
    (dict(batch=0), INVALID, "batch"), (dict(n=-1), INVALID, "sizes"), (dict(nk=(1 << 30) + 1), INVALID, "sizes"),
    (dict(heads=3), INVALID, "heads"), (dict(kv_heads=0), INVALID, "heads"), (dict(heads=0), INVALID, "heads"),
    (dict(heads=1 << 17), INVALID, "heads"), (dict(heads=130, kv_heads=1), UNSUPPORTED, "heads"),
    (dict(dim=0), INVALID, "dim"), (dict(dim=20), UNSUPPORTED, "dim"), (dict(dim=256), UNSUPPORTED, "dim"),
    (dict(scale=0.0), INVALID, "scale"), (dict(scale=-1.0), INVALID, "scale"), (dict(scale=math.nan), INVALID, "scale"),
    (dict(scale=math.inf), INVALID, "scale"), (dict(scale=2e38), INVALID, "scale"),
    (dict(q_start=P + 2), INVALID, "q_start"),
    (dict(k_start=P + 1), INVALID, "k_start"), (dict(k_len=P + 3), INVALID, "k_len"),
    (dict(ALONE, n=1 << 30, nk=1 << 17, causal=0), UNSUPPORTED, "2^31"),
    (dict(ALONE, n=1 << 20, nk=1 << 30), UNSUPPORTED, "2^31"),
    (dict(q_start=None), INVALID, "q_start"), (dict(k_start=None), INVALID, "k_start"), (dict(), INVALID, "handle"),
]


def pitched(name, rows=True):
    return [(dict({name: None}), INVALID, name), (dict({name: P + 8}), INVALID, name),
            (dict({"ld" + name: 8}), INVALID, name), (dict({"h" + name: 15}), INVALID, name),
            (dict({"ld" + name: 68}), UNSUPPORTED, name), (dict({"h" + name: 20}), UNSUPPORTED, name)]


def tensors(names):
    a = {}
    for x in names:
        a.update({x: P, "ld" + x: 64, "h" + x: 16})
    return a


@pytest.mark.parametrize("kw,status,word", COMMON + [c for x in ("q", "k", "v", "out") for c in pitched(x)] +
                         [(dict(lse=P + 2), INVALID, "lse")])
def test_attention_refuses(lib, kw, status, word):
    a = dict(SHAPE, **tensors(("q", "k", "v", "out")), lse=None)
    a.update(kw)
    assert lib.tpo_attention(None, *a.values(), None) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,status,word", COMMON + [c for x in ("dout", "q", "k", "v", "out", "dq", "dk", "dv")
                                                     for c in pitched(x)] +
                         [(dict(lse=P + 2), INVALID, "lse"), (dict(lse=None), INVALID, "lse")])
def test_attention_bwd_refuses(lib, kw, status, word):
    a = dict(SHAPE, **tensors(("dout", "q", "k", "v", "out")), lse=P, **tensors(("dq", "dk", "dv")))
    a.update(kw)
    assert lib.tpo_attention_bwd(None, *a.values(), None) == status
    assert word in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw", [
    dict(ALONE, n=1 << 20, nk=1 << 20, heads=32, kv_heads=8),
    dict(ALONE, n=1 << 17, nk=1 << 22, heads=8, kv_heads=8),
    dict(batch=1 << 20, n=1 << 20, nk=1 << 26, heads=8, kv_heads=1),  # of a few keys each
    dict(ALONE, n=1 << 30, nk=0, heads=1, kv_heads=1, causal=0)])
def test_long_sequences_are_taken(lib, kw):
    """Sizes whose steps 32 bits do count get as far as the handle."""
    a = dict(SHAPE, dim=128)
    a.update(kw)
    heads, kv = a["heads"] * 128, a["kv_heads"] * 128
    q, k = {"ld": heads, "h": 128}, {"ld": kv, "h": 128}

    def of(names):
        out = {}
        for x in names:
            at = q if x in ("q", "out", "dout", "dq") else k
            out.update({x: P, "ld" + x: at["ld"], "h" + x: at["h"]})
        return out

    assert lib.tpo_attention(None, *a.values(), *of(("q", "k", "v", "out")).values(), None, None) == INVALID
    assert "handle" in t.tpo_last_error(), t.tpo_last_error()
    bwd = of(("dout", "q", "k", "v", "out")), of(("dq", "dk", "dv"))
    assert lib.tpo_attention_bwd(None, *a.values(), *bwd[0].values(), P, *bwd[1].values(), None) == INVALID
    assert "handle" in t.tpo_last_error(), t.tpo_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(n=-1), "sizes"), (dict(heads=0), "sizes"), (dict(dim=0), "sizes"), (dict(dim=10000), "sizes"),
    (dict(ny=-1), "sizes"), (dict(rot=3), "rot"), (dict(rot=18), "rot"), (dict(rot=-2), "rot"), (dict(dtype=1), "types"),
    (dict(layout=2), "layout"), (dict(magnitude=math.nan), "magnitude"), (dict(rows=None, ny=5), "ny"),
    (dict(x=None), "x"), (dict(x=P + 1), "x"), (dict(ldx=8), "x"), (dict(hx=8), "x"), (dict(y=None), "y"),
    (dict(dtype=2, y=P + 2), "y"), (dict(hy=1), "y"), (dict(pos=P + 2), "pos"), (dict(rows=P + 1), "rows"),
    (dict(table=None), "table"), (dict(table=P + 4), "table"), (dict(y=P), "y may be x"),
    (dict(y=P, rows=None, ny=4, ldy=128), "y may be x"), (dict(), "handle")])
def test_rotary_refuses(lib, kw, word):
    a = dict(n=4, heads=3, dim=16, rot=8, dtype=0, layout=0, inverse=0, magnitude=1.0, pos=P, table=P, x=P, ldx=48,
             hx=16, rows=P, ny=9, y=2 * P, ldy=48, hy=16)
    a.update(kw)
    assert lib.tpo_rotary(None, *a.values(), None) == INVALID
    assert word in t.tpo_last_error(), t.tpo_last_error()


def test_empty_tensors_need_no_address(lib):
    a = dict(SHAPE, **tensors(("q", "k", "v", "out")), lse=None)
    a.update(n=0, nk=0, q=None, k=None, v=None, out=None)
    assert lib.tpo_attention(None, *a.values(), None) == INVALID
    assert "handle" in t.tpo_last_error()


def test_binding_refuses_host_tensors_types_and_shapes(lib):
    b16 = torch.bfloat16
    q, k = torch.zeros(4, 4, 16, dtype=b16), torch.zeros(6, 2, 16, dtype=b16)
    with pytest.raises(t.TpoError, match="CUDA"):
        t.tpo_attention(1, q, k, k, q)
    with pytest.raises(t.TpoError, match="3-D"):
        t.tpo_attention(1, q[0], k, k, q)
    with pytest.raises(t.TpoError, match="int32"):
        t.tpo_attention(1, q, k, k, q, q_start=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(t.TpoError, match="contiguous elements"):
        t.tpo_attention(1, q, k, k, q, k_len=torch.zeros(1, dtype=torch.int32),
                        k_start=torch.zeros(7, dtype=torch.int32))
    with pytest.raises(t.TpoError, match="CUDA"):
        t.tpo_rotary(1, q, torch.zeros(4, dtype=torch.int64), q)
    with pytest.raises(t.TpoError, match="type"):
        t.tpo_rotary(1, q.double(), None, q)


# ------------------------------------------------------------------ the references

def _directional(f, grads, inputs, gen):
    for name, g in grads.items():
        d = torch.randn(inputs[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        up, down = dict(inputs), dict(inputs)
        up[name], down[name] = inputs[name] + h * d, inputs[name] - h * d
        diff = (f(**up) - f(**down)) / (2 * h)
        assert abs(float((g * d).sum() - diff)) <= 1e-6 * (1 + abs(float(diff))), name


@pytest.mark.parametrize("causal", [False, True])
def test_reference_gradients_against_differences(causal):
    gen = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    seqs = [(0, 4, 0, 6), (4, 3, 6, 3), (7, 2, 9, 1), (9, 1, 10, 0)]
    q, k, v, dout = r(10, 6, 8), r(10, 2, 8), r(10, 2, 8), r(10, 6, 8)
    f = A.attention(q, k, v, seqs, causal, 0.3)
    g = A.attention_bwd(dout, q, k, v, f["out"][0], f["lse"][0], seqs, causal, 0.3)
    _directional(lambda q, k, v: (A.attention(q, k, v, seqs, causal, 0.3)["out"][0] * dout).sum(),
                 dict(q=g["dq"][0], k=g["dk"][0], v=g["dv"][0]), dict(q=q, k=k, v=v), gen)


@pytest.mark.parametrize("pairs", [False, True])
def test_reference_rotary_keeps_differences_of_positions(pairs):
    """<turn(a, i), turn(b, j)> depends on i - j alone, and the inverse undoes the turn."""
    gen = torch.Generator().manual_seed(7)
    a, b = (torch.randn(1, 1, 16, generator=gen, dtype=torch.float64) for _ in range(2))
    freq = A.frequencies(12, 10000.0)
    turn = lambda x, i, **kw: A.rotary(x, torch.tensor([i]), freq, pairs, **kw)[0]  # noqa: E731
    one, two = (turn(a, 7) * turn(b, 3)).sum(), (turn(a, 107) * turn(b, 103)).sum()
    assert abs(float(one - two)) < 1e-9
    assert torch.allclose(turn(turn(a, 9, magnitude=2.0), 9, inverse=True, magnitude=0.5), a)


def test_check_sees_planted_mistakes():
    """The bounds see one key left out of a row, one too many, and a weight's gradient without its delta."""
    gen = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=gen).bfloat16().double()  # noqa: E731
    q, k, v, dout = r(40, 2, 32), r(40, 1, 32), r(40, 1, 32), r(40, 2, 32)
    seqs = [(0, 40, 0, 40)]
    f = A.attention(q, k, v, seqs, True, 0.2)
    out, lse = f["out"][0].bfloat16(), f["lse"][0].float()
    R.check("out", out, f["out"])
    R.check("lse", lse, f["lse"])
    for wrong in ([(0, 40, 0, 39)], [(0, 39, 0, 40)]):
        bad = A.attention(q, k, v, wrong, True, 0.2)["out"][0]
        with pytest.raises(AssertionError):
            R.check("out", bad[:39].bfloat16(), tuple(x[:39] for x in f["out"]))
    g = A.attention_bwd(dout, q, k, v, out.double(), lse.double(), seqs, True, 0.2)
    for name in ("dq", "dk", "dv"):
        R.check(name, g[name][0].bfloat16(), g[name])
    bad = A.attention_bwd(dout, q, k, v, 0 * out.double(), lse.double(), seqs, True, 0.2)
    for name in ("dq", "dk"):
        with pytest.raises(AssertionError):
            R.check(name, bad[name][0].bfloat16(), g[name])
