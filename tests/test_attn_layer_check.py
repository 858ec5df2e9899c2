"""What the attention layer's --check sees of a step of single tokens: a step in
the operators' roundings passes, one with a mistake does not (no GPU)."""

import types

import pytest
import torch

from tensor_comm_gemm_gb300 import attn_layer as L

BF16 = torch.bfloat16
TOL = 4 * 2.0 ** -8  # that of the example's tests


def layer_of(hidden, heads, kv, dim, tp, tokens, cache, gen):
    r = lambda *s, scale=1.0: (torch.randn(*s, generator=gen) * scale).to(BF16)  # noqa: E731
    width = (heads + 2 * kv) // tp * dim
    layer = types.SimpleNamespace(
        hidden=hidden, heads=heads // tp, kv=kv // tp, dim=dim, tp=tp, cache=cache, gamma=(1 + r(hidden, scale=0.1)).to(BF16),
        beta=r(hidden, scale=0.1), wqkv=[r(width, hidden, scale=hidden ** -0.5) for _ in range(tp)],
        wo=[r(hidden, heads // tp * dim, scale=(heads * dim) ** -0.5) for _ in range(tp)],
        k=[r(tokens * cache, kv // tp, dim) for _ in range(tp)], v=[r(tokens * cache, kv // tp, dim) for _ in range(tp)])
    layer.slices = types.MethodType(L.AttnLayer.slices, layer)
    return layer


def step(layer, x, pos, lens, rows, mistake=None):
    """decode(), with each result rounded as the operators round it."""
    n, group = len(x), layer.heads // layer.kv
    norm = torch.nn.functional.layer_norm(x.double(), (layer.hidden,), layer.gamma.double(), layer.beta.double(), L.EPS).to(BF16)
    outs = []
    for r, w in enumerate(layer.wqkv):
        q, k, v = layer.slices((norm.double() @ w.double().T).to(BF16).view(n, -1, layer.dim))
        q = L._turn(q.double(), pos).to(BF16)
        k = k if mistake == "not turned" else L._turn(k.double(), pos).to(BF16)
        to = rows.roll(1) if mistake == "another's row" else rows - 1 if mistake == "a row before" else rows
        if mistake != "not written":
            layer.k[r][to], layer.v[r][to] = k, -v if mistake == "negated" else v
        out = torch.empty_like(q)
        for i, count in enumerate(lens):
            count -= mistake == "a key short"
            at = i * layer.cache
            ks, vs = (c[r][at:at + count].double().repeat_interleave(group, 1) for c in (layer.k, layer.v))
            p = (torch.einsum("hd,khd->hk", q[i].double(), ks) * layer.dim ** -0.5).softmax(1)
            out[i] = torch.einsum("hk,khd->hd", p, vs).to(BF16)
        outs.append(out)
    y = x.double() + torch.cat([o.flatten(1) for o in outs], 1).double() @ torch.cat(layer.wo, 1).double().T
    return dict(y=y.to(BF16), out=outs)


@pytest.mark.parametrize("mistake", [None, "not written", "not turned", "a key short", "another's row", "a row before",
                                     "negated"])
@pytest.mark.parametrize("tokens,hidden,heads,kv,dim,tp,cache", [
    (1, 512, 8, 2, 128, 1, 700), (9, 256, 6, 2, 40, 1, 130), (4, 512, 8, 2, 128, 2, 300)])
def test_check_sees_mistakes_of_a_step(tokens, hidden, heads, kv, dim, tp, cache, mistake):
    gen = torch.Generator().manual_seed(61)
    layer = layer_of(hidden, heads, kv, dim, tp, tokens, cache, gen)
    x = torch.randn(tokens, hidden, generator=gen).to(BF16)
    lens = [cache - 5 * i for i in range(tokens)]
    pos, rows = torch.tensor(lens) - 1, torch.tensor([i * cache + n - 1 for i, n in enumerate(lens)])
    old = [c.clone() for c in layer.k], [c.clone() for c in layer.v]
    errors = L.compare(layer, step(layer, x, pos, lens, rows, mistake), L.reference(layer, x, pos, lens, None, old), rows, old)
    assert set(errors) == {"y", "out", "k", "v", "other rows of k", "other rows of v"}
    if mistake is None or (mistake == "another's row" and tokens == 1):
        assert all(e < TOL for e in errors.values()), errors
    else:
        assert not all(e < TOL for e in errors.values()), errors
        assert errors["y"] < TOL or mistake != "not turned"  # the output with its residual does not show it
