"""The attention sublayer's operators together, as a layer uses them: packed
prompts, training steps, single tokens over a cache and heads shared by ranks."""

import pytest

import block_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built(cuda_ok):
    import __graft_entry__
    __graft_entry__.build()


# The stages' roundings to bf16 (norm, qkv, the turned q and k, weights, out; backward dout, ds, dqkv turned, dnorm) are
# about ten of at most 2^-8 of each result's size, spread evenly: together about 2^-8 / sqrt(3) * sqrt(10), below 2 * 2^-8.
@pytest.mark.parametrize("args", [
    "--tokens 300 --hidden 256 --heads 4 --kv-heads 2 --dim 64 --sequences 3 --train",
    "--tokens 517 --hidden 512 --heads 8 --kv-heads 1 --train",
    "--tokens 256 --hidden 320 --heads 3 --kv-heads 3 --dim 80",
    "--tokens 512 --hidden 256 --heads 8 --kv-heads 4 --dim 64 --tp 2 --sequences 2",
    "--tokens 1 --hidden 512 --heads 8 --kv-heads 2 --cache 700",
    "--tokens 9 --hidden 256 --heads 6 --kv-heads 2 --dim 40 --cache 130",
    "--tokens 4 --hidden 512 --heads 8 --kv-heads 2 --cache 300 --tp 2"])
def test_example_layer(args):
    from tensor_comm_gemm_gb300 import attn_layer
    errors = attn_layer.main(args.split() + ["--check", "--calls", "2"])
    assert errors and all(e < 4 * R.U16 for e in errors.values()), errors


def test_example_refuses():
    from tensor_comm_gemm_gb300 import attn_layer
    with pytest.raises(ValueError):
        attn_layer.AttnLayer(256, 4, 2, 64, tp=4)
    with pytest.raises(ValueError):
        attn_layer.AttnLayer(256, 4, 2, 64, cache=10, train=True)
