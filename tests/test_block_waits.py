"""The bound of the block operators' device-side waits: the option, and calls
whose waits run out."""

import pytest

from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


@pytest.mark.parametrize("value,word", [(0, "wait_timeout_ms"), (-1, "wait_timeout_ms"), (600001, "wait_timeout_ms"),
                                        (1, "handle"), (600000, "handle")])
def test_option_range(lib, value, word):
    assert lib.tpo_block_set_opt(None, b"wait_timeout_ms", value) == t.TPO_ERR_INVALID_ARG
    assert word in t.tpo_last_error()


@pytest.mark.gpu
def test_option_round_trip(cuda_ok, lib):
    b = t.tpo_block_create(0)
    try:
        assert t.tpo_block_get_opt(b, "wait_timeout_ms") == 2000
        t.tpo_block_set_opt(b, "wait_timeout_ms", 50)
        assert t.tpo_block_get_opt(b, "wait_timeout_ms") == 50
        assert t.tpo_block_get_opt(b, "path") == 0 and t.tpo_block_get_opt(b, "split") == 0
    finally:
        t.tpo_block_destroy(b)


# ------------------------------------------------------------------ waits that run out
#
# A contraction of a million terms and more keeps the epilogue waiting for
# several milliseconds: with a bound of one it gives up, with MMAs and loads in
# flight.  The call then reports the failure once, and the handle goes on.

def _linear(torch, rnd, n, k, m, dtype=None):
    x, w, y = rnd(n, k), rnd(m, k), torch.empty(n, m, dtype=torch.bfloat16, device="cuda")
    s = None
    if dtype is not None:
        x, w, s = x.to(dtype), w.to(dtype), torch.ones(1, device="cuda")
    return lambda b: t.tpo_linear(b, x, w, y, act=t.TPO_ACT_SILU, scale_inv_x=s, scale_inv_w=s), [y]


def _gated(torch, rnd, n, k, m):
    x, wg, wu, h = rnd(n, k), rnd(m, k), rnd(m, k), torch.empty(n, m, dtype=torch.bfloat16, device="cuda")
    return lambda b: t.tpo_gated(b, x, wg, wu, h), [h]


def _linear_bwd(torch, rnd, n, k, m):
    dy, x, w = rnd(n, m), rnd(n, k), rnd(m, k)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    return lambda b: t.tpo_linear_bwd(b, dy, x, w, dx=dx, dw=dw), [dx, dw]


def _gated_bwd(torch, rnd, n, k, m):
    dh, g, u, x, wg, wu = rnd(n, m), rnd(n, m), rnd(n, m), rnd(n, k), rnd(m, k), rnd(m, k)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    return lambda b: t.tpo_gated_bwd(b, dh, g, u, x, wg, wu, dx=dx, dwg=dwg, dwu=dwu), [dx, dwg, dwu]


LONG = {
    "linear on pairs": (1, 0, lambda c, r: _linear(c, r, 300, 1 << 20, 520)),
    "linear e4m3 on pairs": (1, 0, lambda c, r: _linear(c, r, 256, 1 << 21, 256, c.float8_e4m3fn)),
    "gated on pairs": (1, 0, lambda c, r: _gated(c, r, 256, 1 << 20, 136)),
    "linear gradients on pairs": (1, 0, lambda c, r: _linear_bwd(c, r, 1 << 20, 136, 72)),
    "gated gradients on pairs": (1, 0, lambda c, r: _gated_bwd(c, r, 1 << 20, 64, 64)),
    "linear on one CTA": (2, 1, lambda c, r: _linear(c, r, 16, 1 << 20, 264)),
    "linear on clusters": (2, 8, lambda c, r: _linear(c, r, 100, 1 << 22, 128)),
    "gated on clusters": (2, 2, lambda c, r: _gated(c, r, 9, 1 << 21, 72)),
    "linear gradients on clusters": (2, 2, lambda c, r: _linear_bwd(c, r, 1 << 21, 64, 72)),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", LONG)
def test_wait_that_runs_out_is_reported_once(cuda_ok, lib, name):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    path, split, make = LONG[name]
    run, outs = make(torch, rnd)
    b = t.tpo_block_create(t.tpo_block_workspace(t.TPO_OP_GATED_BWD, 1 << 20, 64, 64) if "gated grad" in name else 0)
    try:
        t.tpo_block_set_opt(b, "path", path)
        t.tpo_block_set_opt(b, "split", split)
        run(b)
        assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
        first = [o.clone() for o in outs]
        assert all(torch.isfinite(o).all() for o in first)
        for _ in range(6):
            t.tpo_block_set_opt(b, "wait_timeout_ms", 1)
            run(b)
            assert t.tpo_block_sync_status(b) == 4
            assert "timed out" in t.tpo_last_error()
            assert t.tpo_block_sync_status(b) == 0
            t.tpo_block_set_opt(b, "wait_timeout_ms", 2000)
            for o in outs:
                o.zero_()
            run(b)
            assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
            assert all(torch.equal(o, f) for o, f in zip(outs, first))
    finally:
        t.tpo_block_destroy(b)
