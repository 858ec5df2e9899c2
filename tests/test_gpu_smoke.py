"""smoke() fails if either layer's results are off, whatever the other's are."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wrong", ["ffn_layer", "attn_layer"])
def test_smoke_sees_each_layer(cuda_ok, monkeypatch, wrong):
    import __graft_entry__ as g
    from tensor_comm_gemm_gb300 import attn_layer, ffn_layer
    g.build()
    for layer in (ffn_layer, attn_layer):
        bad = layer.__name__.endswith(wrong)
        monkeypatch.setattr(layer, "main", lambda argv, bad=bad: dict(y=0.5 if bad else 0.001, dx=0.001))
    with pytest.raises(AssertionError, match="0.5"):
        g.smoke()
