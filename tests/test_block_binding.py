"""Arguments of the block operators' Python calls that a call does not need."""

import pytest
import torch

import block_ref as R
from tensor_comm_gemm_gb300 import build as tb
from tensor_comm_gemm_gb300 import tpoverlap as t

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    tb.build()
    return t.lib()


def test_gated_gradients_take_their_width_from_any_matrix(lib):
    dh, w = torch.zeros(4, 8, dtype=BF16), torch.zeros(8, 16, dtype=BF16)
    # refused for being host tensors, not for the matrices that are not there
    with pytest.raises(t.TpoError, match="dh must be a CUDA tensor"):
        t.tpo_gated_bwd(1, dh, dh, dh, None, w, w, dx=torch.zeros(4, 16, dtype=BF16))
    with pytest.raises(t.TpoError, match="2-D"):
        t.tpo_gated_bwd(1, dh, dh, dh, None, w[0], w)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["dx", "dw", "none"])
def test_gated_gradients_without_what_they_do_not_need(cuda_ok, lib, which):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    n, k, m = 70, 136, 200
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)  # noqa: E731
    dh, g, u, x, wg, wu = r(n, m), r(n, m), r(n, m), r(n, k), r(m, k), r(m, k)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    b = t.tpo_block_create(t.tpo_block_workspace(t.TPO_OP_GATED_BWD, n, k, m))
    try:
        if which == "dx":
            t.tpo_gated_bwd(b, dh, g, u, None, wg, wu, dx=dx)
        elif which == "dw":
            t.tpo_gated_bwd(b, dh, g, u, x, None, None, dwg=dwg, dwu=dwu)
        else:
            t.tpo_gated_bwd(b, dh, g, u, None, None, None)
        assert t.tpo_block_sync_status(b) == 0, t.tpo_last_error()
    finally:
        t.tpo_block_destroy(b)
    want = R.gated_bwd(*(v.double() for v in (dh, g, u, x, wg, wu)))
    if which == "dx":
        R.check("dx", dx, want["dx"])
    if which == "dw":
        R.check("dwg", dwg, want["dwg"])
        R.check("dwu", dwu, want["dwu"])
