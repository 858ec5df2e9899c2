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
