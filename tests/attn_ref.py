"""References of the attention sublayer's operators in 64 bits, and how far a
computed output may be from them (see block_ref for the form and the bounds of
sums).  Sequences are given as (first query row, queries, first key row, keys).

Weights: a score is a sum of dim products in fp32, and its error is the relative
error of its exponential; the exponential and its argument add a few 2^-24 of
the argument's size.  The weights (and the scores' gradients) are rounded to
bf16, 2^-8 of each, as operands of the products that follow.
"""

import math

import torch

from block_ref import U16, U32, _sum_slack

INF = math.inf


def sees(nq, nk, causal, device):
    """[nq, nk]: whether query i sees key j."""
    i, j = torch.arange(nq, device=device)[:, None], torch.arange(nk, device=device)[None]
    return j <= i + (nk - nq) if causal else (j >= 0) & (i >= 0)


def _scores(q, k, scale, mask):
    z = (q @ k.T) * scale
    slack = _sum_slack(q.shape[1], q.abs() @ k.abs().T) * scale
    return z.masked_fill(~mask, -INF), slack.masked_fill(~mask, 0.0)


def _attend(q, k, v, scale, mask):
    """One head of one sequence: out, lse and their slacks."""
    z, sz = _scores(q, k, scale, mask)
    any_key = mask.any(1)
    top = torch.where(any_key, z.amax(1) if z.shape[1] else z.new_zeros(len(z)), z.new_zeros(len(z)))
    p = torch.exp(z - top[:, None]).masked_fill(~mask, 0.0)
    total = p.sum(1)
    w = p / torch.where(any_key, total, torch.ones_like(total))[:, None]
    out = w @ v
    size = torch.where(mask, z.abs(), 0.0) + top.abs()[:, None] + 1
    rel = sz + 16 * U32 * size  # of one weight
    mean = (w * rel).sum(1)     # of their sum
    keys = mask.sum(1).double()
    s_out = (w * (rel + U16)) @ v.abs() + (mean + (keys + 16) * 2 * U32)[:, None] * (w @ v.abs())
    lse = torch.where(any_key, top + torch.log(total), torch.full_like(top, -INF))
    s_lse = mean + (keys + 16) * 2 * U32 + 8 * U32 * (lse.abs() + 1)
    return out, s_out, lse, torch.where(any_key, s_lse, torch.zeros_like(s_lse))


def attention(q, k, v, seqs, causal, scale):
    """{out: ([n, heads, dim], slack), lse: ([n, heads], slack)}; rows of no sequence are NaN."""
    n, heads, _ = q.shape
    group = heads // k.shape[1]
    out, s_out = torch.full_like(q, math.nan), torch.zeros_like(q)
    lse, s_lse = out[:, :, 0].clone(), s_out[:, :, 0].clone()
    for q0, nq, k0, nk in seqs:
        mask = sees(nq, nk, causal, q.device)
        for h in range(heads):
            o = _attend(q[q0:q0 + nq, h], k[k0:k0 + nk, h // group], v[k0:k0 + nk, h // group], scale, mask)
            for t, x in zip((out, s_out, lse, s_lse), o):
                t[q0:q0 + nq, h] = x
    return dict(out=(out, s_out), lse=(lse, s_lse))


def attention_bwd(dout, q, k, v, out, lse, seqs, causal, scale):
    """Gradients by the formula from the given out and lse, and their slacks; rows of no sequence are NaN."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    g = {x: torch.full_like(t, math.nan) for x, t in (("dq", q), ("dk", k), ("dv", v))}
    s = {x: torch.zeros_like(t) for x, t in g.items()}
    for q0, nq, k0, nk in seqs:
        mask = sees(nq, nk, causal, q.device)
        rq, rk = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for t in (g, s):
            t["dq"][rq], t["dk"][rk], t["dv"][rk] = 0.0, 0.0, 0.0
        for h in range(heads):
            c = h // group
            qh, kh, vh, doh = q[rq, h], k[rk, c], v[rk, c], dout[rq, h]
            z, sz = _scores(qh, kh, scale, mask)
            known = torch.where(lse[rq, h] == -INF, 0.0, lse[rq, h])[:, None]
            p = torch.exp(z - known).masked_fill(~mask, 0.0)
            rel = sz + 16 * U32 * (torch.where(mask, z.abs(), 0.0) + known.abs() + 1)
            dp, s_dp = doh @ vh.T, _sum_slack(dim, doh.abs() @ vh.abs().T)
            delta = (doh * out[rq, h]).sum(1, keepdim=True)
            s_delta = _sum_slack(dim, (doh * out[rq, h]).abs().sum(1, keepdim=True))
            ds = p * (dp - delta)
            s_ds = ds.abs() * (rel + 4 * U32) + p * (s_dp + s_delta + 2 * U32 * (dp.abs() + delta.abs())) * (1 + rel)
            s_ds = s_ds + U16 * (ds.abs() + s_ds)
            s_p = p * (rel + U16)
            g["dq"][rq, h] = scale * (ds @ kh)
            s["dq"][rq, h] = scale * (s_ds @ kh.abs() + _sum_slack(nk, ds.abs() @ kh.abs()))
            g["dk"][rk, c] += scale * (ds.T @ qh)
            s["dk"][rk, c] += scale * (s_ds.T @ qh.abs() + _sum_slack(nq * group, ds.abs().T @ qh.abs()))
            g["dv"][rk, c] += p.T @ doh
            s["dv"][rk, c] += s_p.T @ doh.abs() + _sum_slack(nq * group, p.T @ doh.abs())
    return {x: (g[x], s[x]) for x in g}


def frequencies(rot, base, scaling="none", factor=1.0, low=1.0, high=4.0, original=1):
    """Radians a position of each pair."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f *= keep + (1 - keep) / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rotary(x, pos, freq, pairs=False, inverse=False, magnitude=1.0):
    """(y, slack): the angle's 2^-26 turns and the fp32 sine, cosine, products and sum."""
    rot = 2 * len(freq)
    t = pos.double()[:, None] * freq.to(x.device)
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None] * (-1 if inverse else 1)
    ia = torch.arange(0, rot, 2) if pairs else torch.arange(rot // 2)
    ib = ia + 1 if pairs else ia + rot // 2
    a, b = x[..., ia], x[..., ib]
    y, slack = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = magnitude * (a * c - b * s), magnitude * (a * s + b * c)
    # 64-bit products of far positions are themselves off by 2^-53 of the angle
    off = 2 * math.pi * 2.0 ** -25 + 8 * U32 + 2.0 ** -51 * (t.abs().max().item() if t.numel() else 0.0)
    slack[..., ia] = slack[..., ib] = abs(magnitude) * off * (a.abs() + b.abs())
    return y, slack
