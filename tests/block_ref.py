"""References of the block operators in 64 bits, and how far a computed output
may be from them.

Every function returns {name: (value, slack)}: the operator's definition in
64 bits and a bound on the error of its computation in fp32, element by
element, before the output's own rounding.  The bounds follow from the
formulas: a sum of K terms carried in fp32 is off by at most about
K 2^-23 times the sum of the terms' magnitudes (2^-24 for each rounding, twice
that for an accumulator that truncates); a value rounded to bf16 by 2^-8 of
itself; a value of an fp32 function by a few 2^-24 of its arguments' size.
"""

import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24  # half a unit in the last of 8 and of 24 bits
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LIP = 1.2  # the activations' largest slope is about 1.13


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


def _sum_slack(terms, magnitude):
    return (terms + 16) * 2 * U32 * magnitude


def product(a, b):
    """a b^T in 64 bits and its fp32 slack."""
    return a @ b.T, _sum_slack(a.shape[1], a.abs() @ b.abs().T)


def linear(x, w, bias=None, act_name="none", residual=None, scale=1.0):
    z, s = product(x, w)
    z, s = z * scale, (s + 4 * U32 * z.abs()) * scale
    if bias is not None:
        z = z + bias
        s = s + U32 * z.abs()
    y = act(z, act_name)
    sy = LIP * s + 64 * U32 * (z.abs() + 1) * (act_name not in ("none", "relu"))
    if residual is not None:
        y = y + residual
        sy = sy + U32 * y.abs()
    return dict(y=(y, sy), z=(z, s))


def linear_bwd(dy, x, w, z=None, act_name="none"):
    d = dy if z is None else dy * act_grad(z, act_name)
    # the derivative in fp32; dz is a matrix operand, so it is rounded to bf16 unless it is dy itself
    sd = 0 * d if z is None else 64 * U32 * dy.abs() * (1 + (z.abs() if z is not None else 0))
    so = sd if z is None else sd + U16 * (d.abs() + sd)
    dx, s1 = product(d, w.T)
    dw, s2 = product(d.T, x.T)
    db = d.sum(0)
    return dict(dx=(dx, s1 + so @ w.abs()), dw=(dw, s2 + so.T @ x.abs()),
                db=(db, _sum_slack(d.shape[0], d.abs().sum(0)) + sd.sum(0)))


def gated(x, wg, wu, act_name="silu", scale_g=1.0, scale_u=1.0):
    g, sg = product(x, wg)
    u, su = product(x, wu)
    g, sg = g * scale_g, (sg + 4 * U32 * g.abs()) * scale_g
    u, su = u * scale_u, (su + 4 * U32 * u.abs()) * scale_u
    a = act(g, act_name)
    sa = LIP * sg + 64 * U32 * (g.abs() + 1) * (act_name not in ("none", "relu"))
    h = a * u
    return dict(h=(h, sa * u.abs() + a.abs() * su + sa * su + U32 * h.abs()), g=(g, sg), u=(u, su))


def gated_bwd(dh, g, u, x, wg, wu, act_name="silu"):
    dg, du = dh * u * act_grad(g, act_name), dh * act(g, act_name)
    fn = 64 * U32 * (1 + g.abs())
    sg = fn * (dh * u).abs()
    su = fn * dh.abs()
    sg, su = sg + U16 * (dg.abs() + sg), su + U16 * (du.abs() + su)  # both are matrix operands in bf16
    a, s1 = product(dg, wg.T)
    b, s2 = product(du, wu.T)
    dwg, s3 = product(dg.T, x.T)
    dwu, s4 = product(du.T, x.T)
    # dx is one chain of 2 m terms
    s12 = 2 * (s1 + s2) + sg @ wg.abs() + su @ wu.abs()
    return dict(dx=(a + b, s12), dwg=(dwg, s3 + sg.T @ x.abs()), dwu=(dwu, s4 + su.T @ x.abs()))


def layer_norm(x, gamma, beta, eps):
    k = x.shape[1]
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1 / torch.sqrt((xc * xc).mean(1) + eps)
    xhat = xc * rstd[:, None]
    # sums of k terms by at least 32 lanes, so no chain is longer than k / 32 + 32
    c = (k / 32 + 32) * U32
    s_mean = c * x.abs().mean(1)
    s_xc = s_mean[:, None] + U32 * (x.abs() + mean.abs()[:, None])
    # the variance moves by 2 mean(|xc| s_xc) + mean(s_xc^2) and its own rounding
    s_var = 2 * (xc.abs() * s_xc).mean(1) + (s_xc * s_xc).mean(1) + c / rstd ** 2
    s_rstd = rstd * (0.5 * s_var * rstd ** 2 + 8 * U32)
    g = torch.ones_like(x[0]) if gamma is None else gamma
    b = torch.zeros_like(x[0]) if beta is None else beta
    y = xhat * g + b
    s_hat = rstd[:, None] * s_xc + xc.abs() * s_rstd[:, None] + (s_xc * s_rstd[:, None]) + 4 * U32 * xhat.abs()
    s_y = s_hat * g.abs() + 4 * U32 * ((xhat * g).abs() + b.abs())
    return dict(y=(y, s_y), mean=(mean, s_mean), rstd=(rstd, s_rstd))


def layer_norm_bwd(dy, x, gamma, mean, rstd, dres=None):
    n, k = x.shape
    g = torch.ones_like(x[0]) if gamma is None else gamma
    r = rstd[:, None]
    xhat = (x - mean[:, None]) * r
    s_hat = r * U32 * (x.abs() + mean.abs()[:, None]) + 4 * U32 * xhat.abs()
    a = dy * g
    c = (k / 32 + 32) * U32
    m1, m2 = a.mean(1, keepdim=True), (a * xhat).mean(1, keepdim=True)
    s1 = c * a.abs().mean(1, keepdim=True)
    s2 = (c * (a * xhat).abs() + a.abs() * s_hat).mean(1, keepdim=True)
    dx = r * (a - m1 - xhat * m2)
    s = r * (4 * U32 * (a.abs() + m1.abs() + (xhat * m2).abs()) + s1 + s2 * xhat.abs() + s_hat * (m2.abs() + s2))
    if dres is not None:
        dx = dx + dres
        s = s + U32 * dx.abs()
    return dict(dx=(dx, s + 4 * U32 * dx.abs()),
                dgamma=((dy * xhat).sum(0), _sum_slack(n, (dy * xhat).abs().sum(0)) + (dy.abs() * s_hat).sum(0)),
                dbeta=(dy.sum(0), _sum_slack(n, dy.abs().sum(0))))


def check(name, got, want):
    """got (a tensor of the output's type) is within the fp32 slack and its own rounding of want."""
    ref, slack = want
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    own = {torch.bfloat16: U16, torch.float32: U32}[got.dtype]
    g = got.double()
    bound = slack + own * (ref.abs() + slack) + 1e-37
    finite = torch.isfinite(ref)
    assert torch.isfinite(g[finite]).all(), "%s: non-finite values" % name
    assert (torch.isnan(g) == torch.isnan(ref)).all(), "%s: NaN elsewhere" % name
    err = (g - ref).abs()[finite]
    over = err - bound[finite]
    assert (over <= 0).all(), "%s: %d of %d outside, worst error %.3e (bound %.3e)" % (
        name, int((over > 0).sum()), err.numel(), err[over.argmax()], bound[finite][over.argmax()])
