"""Cases of the transformer block's operators: layer norm, the linear layer with
its epilogue, and the gated feed-forward projections, each forward and backward.

A case names an operator ("op"), a direction ("dir") and sizes:

  norm    x [n, k] -> y [n, k], and its backward pass;
  linear  y [n, m] = act(x [n, k] . w [m, k]^T + bias) + residual, and its backward pass;
  gated   h [n, m] = act(x . wg^T) * (x . wu^T) with wg, wu [m, k], and its backward pass.

n counts tokens, k the input features and m the output features.  "dtype" is the
type of the activations and weights (bf16, e4m3 with one scale per tensor, or
for the norm f32); outputs of the products are bf16.  Weights are those of one
rank of a tensor-parallel layer.  "pad" widens x's rows: x is then a column
slice of a wider buffer, as a projection's input often is.
"""

import math
import weakref

import torch

own = False

EPS = 1e-5
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LARGEST_FLOPS = 8.0 * 8192 * 8192 * 3584
LARGEST_BYTES = 8.0 * 16384 * 4096


def listed():
    return [
        # The norm ahead of a projection while one token is generated: latency only.
        dict(name="norm_token", op="norm", dir="fwd", dtype="bf16", wdtype="bf16", n=1, k=4096),
        # The same norm over a long prompt of a wide model.
        dict(name="norm_prompt", op="norm", dir="fwd", dtype="bf16", wdtype="bf16", n=8192, k=8192),
        # Its backward pass in training, with the residual branch's gradient added.
        dict(name="norm_bwd", op="norm", dir="bwd", dtype="bf16", wdtype="bf16", n=16384, k=4096, dres=True),
        # Full-precision norm of an odd width and row count (an embedding trunk kept in f32).
        dict(name="norm_bwd_f32_odd", op="norm", dir="bwd", dtype="f32", wdtype="f32", n=777, k=5003, dres=False),
        # Attention's output projection for one generated token, added to the residual stream.
        dict(name="linear_token", op="linear", dir="fwd", dtype="bf16", n=1, k=4096, m=4096, act="none", bias=True,
             residual=True, save=False, pad=0),
        # A rank's down projection for a batch of 48 decoding sequences, its input a slice of a wider buffer.
        dict(name="linear_batch", op="linear", dir="fwd", dtype="bf16", n=48, k=3584, m=8192, act="none", bias=False,
             residual=True, save=False, pad=512),
        # First projection of a plain feed-forward layer in training: the pre-activation is kept for the backward pass.
        dict(name="linear_train", op="linear", dir="fwd", dtype="bf16", n=4096, k=4096, m=4096, act="gelu_tanh",
             bias=True, residual=False, save=True, pad=0),
        # A column-parallel projection of a prompt in 8 bits.
        dict(name="linear_e4m3", op="linear", dir="fwd", dtype="e4m3", n=2048, k=8192, m=7168, act="none", bias=True,
             residual=False, save=False, pad=0),
        # Backward pass of linear_train's layer.
        dict(name="linear_bwd", op="linear", dir="bwd", dtype="bf16", n=4096, k=4096, m=4096, act="gelu_tanh",
             bias=True),
        # Gated feed-forward projections of a few decoding sequences.
        dict(name="gated_tokens", op="gated", dir="fwd", dtype="bf16", n=4, k=8192, m=3584, act="silu", save=False,
             pad=0),
        # The same of a prompt of ragged length on a wide layer.
        dict(name="gated_prompt", op="gated", dir="fwd", dtype="bf16", n=1777, k=4096, m=14336, act="silu",
             save=False, pad=0),
        # Training's backward pass of a rank's gated projections; the largest case.
        dict(name="gated_bwd", op="gated", dir="bwd", dtype="bf16", n=8192, k=8192, m=3584, act="silu"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        op = rng.choice(("norm", "linear", "linear", "gated"))
        bwd = rng.random() < 0.4
        c = dict(op=op, dir="bwd" if bwd else "fwd")
        if op == "norm":
            c["dtype"] = rng.choice(("bf16", "bf16", "f32"))
            c["wdtype"] = "f32" if c["dtype"] == "f32" else rng.choice(("bf16", "f32"))
            c["n"] = _log(rng, 1, 16384)
            c["k"] = _log(rng, 64, 16384)
            if rng.random() < 0.6:
                c["k"] = max(64, c["k"] // 8 * 8)
            if bwd:
                c["dres"] = rng.random() < 0.5
        else:
            c["dtype"] = "bf16" if bwd or rng.random() < 0.75 else "e4m3"
            unit = 16 if c["dtype"] == "e4m3" else 8
            c["n"] = _log(rng, 16 if bwd else 1, 8192)
            c["k"] = unit * _log(rng, 256 // unit, 8192 // unit)
            c["m"] = 8 * _log(rng, 32, 1792)
            if op == "linear":
                c["act"] = rng.choice(ACTS)
                c["bias"] = rng.random() < 0.5
                if not bwd:
                    c["residual"] = rng.random() < 0.5
            else:
                c["act"] = rng.choice(ACTS[1:])
            if not bwd:
                c["save"] = rng.random() < 0.3
                c["pad"] = rng.choice((0, 0, unit, 256))
        if 3072 in c.values():  # a width that no configuration of this library has
            continue
        w = work(c)
        if w["flops"] <= LARGEST_FLOPS and (op != "norm" or w["bytes"] <= LARGEST_BYTES):
            return c


def work(case):
    n, k = case["n"], case["k"]
    if case["op"] == "norm":
        e, we = (2 if case["dtype"] == "bf16" else 4), (2 if case["wdtype"] == "bf16" else 4)
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * k * e + 2 * k * we + 8 * n, "flops": 8 * n * k}
        return {"bytes": (4 if case["dres"] else 3) * n * k * e + 3 * k * we + 8 * n, "flops": 14 * n * k}
    m, e = case["m"], (1 if case["dtype"] == "e4m3" else 2)
    if case["op"] == "linear":
        if case["dir"] == "fwd":
            outs = 1 + int(case["residual"]) + int(case["save"])
            return {"bytes": (n * k + m * k) * e + 2 * n * m * outs + 2 * m * int(case["bias"]), "flops": 2 * n * k * m}
        reads = 1 if case["act"] == "none" else 2
        return {"bytes": 4 * n * k + 4 * m * k + 2 * n * m * reads + 2 * m * int(case["bias"]), "flops": 4 * n * k * m}
    if case["dir"] == "fwd":
        return {"bytes": (n * k + 2 * m * k) * e + 2 * n * m * (3 if case["save"] else 1), "flops": 4 * n * k * m}
    return {"bytes": 4 * n * k + 8 * m * k + 6 * n * m, "flops": 8 * n * k * m}


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _inputs(case, seed):
    """The tensors of one case, from its seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 17)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)

    def codes(v):
        """One scale per tensor, its largest value at the format's largest."""
        inv = (v.abs().amax() / 448.0).reshape(1)
        return (v / inv).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn), inv

    def sliced(v, pad):
        """v as the leading columns of a wider buffer."""
        if not pad:
            return v
        wide = torch.zeros(v.shape[0], v.shape[1] + pad, dtype=v.dtype, device="cuda")
        wide[:, : v.shape[1]] = v
        return wide[:, : v.shape[1]]

    n, k = case["n"], case["k"]
    t = {}
    if case["op"] == "norm":
        dt, wt = _TYPES[case["dtype"]], _TYPES[case["wdtype"]]
        # a residual stream: a few channels far larger than the rest, and a small common offset
        channel = 1.0 + 12.0 * (torch.rand(k, generator=gen, device="cuda") < 0.004).float()
        t["x"] = (normal(n, k) * channel + 0.1).to(dt)
        t["gamma"] = (1.0 + normal(k, scale=0.2)).to(wt)
        t["beta"] = normal(k, scale=0.1).to(wt)
        if case["dir"] == "bwd":
            t["dy"] = normal(n, k).to(dt)
            t["dres"] = normal(n, k).to(dt) if case["dres"] else None
            xf = t["x"].double()
            mean = xf.mean(1)
            t["rstd"] = (1.0 / torch.sqrt((xf - mean[:, None]).square().mean(1) + EPS)).float()
            t["mean"] = mean.float()
        return t
    m = case["m"]
    wide = 1.0 / math.sqrt(k)
    x, pad = normal(n, k), case.get("pad", 0)
    names = ["w"] if case["op"] == "linear" else ["wg", "wu"]
    for name in names:
        w = normal(m, k, scale=1.5 * wide)
        if case["dtype"] == "e4m3":
            t[name], t["scale_" + name] = codes(w)
        else:
            t[name], t["scale_" + name] = w.to(torch.bfloat16), None
    if case["dtype"] == "e4m3":
        x, t["scale_x"] = codes(x)
    else:
        x, t["scale_x"] = x.to(torch.bfloat16), None
    t["x"] = sliced(x, pad)
    if case["op"] == "linear":
        t["bias"] = normal(m, scale=0.3).to(torch.bfloat16) if case["bias"] else None
        if case["dir"] == "fwd":
            t["residual"] = normal(n, m).to(torch.bfloat16) if case["residual"] else None
        else:
            t["dy"] = normal(n, m).to(torch.bfloat16)
            z = x @ t["w"].T
            t["z"] = None if case["act"] == "none" else (z + t["bias"] if case["bias"] else z)
    elif case["dir"] == "bwd":
        t["dh"] = normal(n, m).to(torch.bfloat16)
        t["g"], t["u"] = x @ t["wg"].T, x @ t["wu"].T
    return t


class _Block:
    """The operators' handle and its workspace, given back with the state."""

    def __init__(self, binding, op, n, k, m):
        self.handle = binding.tpo_block_create(binding.tpo_block_workspace(op, n, k, m))
        weakref.finalize(self, binding.tpo_block_destroy, self.handle)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=dict(case))
    if not own:
        return s
    from tensor_comm_gemm_gb300 import tpoverlap as t

    n, k, m = case["n"], case["k"], case.get("m", 0)

    def like(shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s["t"] = t
    if case["op"] != "norm":
        s["act"] = {"none": t.TPO_ACT_NONE, "relu": t.TPO_ACT_RELU, "gelu": t.TPO_ACT_GELU,
                    "gelu_tanh": t.TPO_ACT_GELU_TANH, "silu": t.TPO_ACT_SILU}[case["act"]]
    if case["op"] == "norm":
        op = t.TPO_OP_LAYER_NORM if case["dir"] == "fwd" else t.TPO_OP_LAYER_NORM_BWD
        if case["dir"] == "fwd":
            s["out"] = dict(y=like((n, k), s["x"].dtype), mean=like((n,), torch.float32),
                            rstd=like((n,), torch.float32))
        else:
            s["out"] = dict(dx=like((n, k), s["x"].dtype), dgamma=like((k,), s["gamma"].dtype),
                            dbeta=like((k,), s["gamma"].dtype))
    elif case["op"] == "linear":
        op = t.TPO_OP_LINEAR if case["dir"] == "fwd" else t.TPO_OP_LINEAR_BWD
        if case["dir"] == "fwd":
            s["out"] = dict(y=like((n, m)))
            if case["save"]:
                s["out"]["z"] = like((n, m))
        else:
            s["out"] = dict(dx=like((n, k)), dw=like((m, k)))
            if case["bias"]:
                s["out"]["db"] = like((m,))
    else:
        op = t.TPO_OP_GATED if case["dir"] == "fwd" else t.TPO_OP_GATED_BWD
        if case["dir"] == "fwd":
            s["out"] = dict(h=like((n, m)))
            if case["save"]:
                s["out"].update(g=like((n, m)), u=like((n, m)))
        else:
            s["out"] = dict(dx=like((n, k)), dwg=like((m, k)), dwu=like((m, k)))
    s["block"] = _Block(t, op, n, k, m)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    t, c, o, block = s["t"], s["case"], s["out"], s["block"].handle
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            t.tpo_layer_norm(block, s["x"], s["gamma"], s["beta"], o["y"], mean=o["mean"], rstd=o["rstd"], eps=EPS)
        else:
            t.tpo_layer_norm_bwd(block, s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], o["dx"],
                                 dgamma=o["dgamma"], dbeta=o["dbeta"], dres=s["dres"])
    elif c["op"] == "linear":
        if c["dir"] == "fwd":
            t.tpo_linear(block, s["x"], s["w"], o["y"], bias=s["bias"], act=s["act"], residual=s["residual"],
                         z=o.get("z"), scale_inv_x=s["scale_x"], scale_inv_w=s["scale_w"])
        else:
            t.tpo_linear_bwd(block, s["dy"], s["x"], s["w"], o["dx"], o["dw"], db=o.get("db"), act=s["act"],
                             z=s["z"])
    elif c["dir"] == "fwd":
        t.tpo_gated(block, s["x"], s["wg"], s["wu"], o["h"], act=s["act"], g=o.get("g"), u=o.get("u"),
                    scale_inv_x=s["scale_x"], scale_inv_wg=s["scale_wg"], scale_inv_wu=s["scale_wu"])
    else:
        t.tpo_gated_bwd(block, s["dh"], s["g"], s["u"], s["x"], s["wg"], s["wu"], o["dx"], o["dwg"], o["dwu"],
                        act=s["act"])
    return o


_R2PI, _C3 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_R2PI * (z + _C3 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        th = torch.tanh(_R2PI * (z + _C3 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * _R2PI * (1 + 3 * _C3 * z * z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


def _product(s, name):
    z = s["x"].float() @ s[name].float().T
    return z if s["scale_x"] is None else z * (s["scale_x"] * s["scale_" + name])


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        x, gamma = s["x"].float(), s["gamma"].float()
        if c["dir"] == "fwd":
            mean = x.mean(1)
            xc = x - mean[:, None]
            rstd = 1 / torch.sqrt((xc * xc).mean(1) + EPS)
            y = xc * rstd[:, None] * gamma + s["beta"].float()
            return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (x - s["mean"][:, None]) * rstd
        a = dy * gamma
        dx = rstd * (a - a.mean(1, keepdim=True) - xhat * (a * xhat).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        wt = s["gamma"].dtype
        return dict(dx=dx.to(s["x"].dtype), dgamma=(dy * xhat).sum(0).to(wt), dbeta=dy.sum(0).to(wt))
    bf16 = torch.bfloat16
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            z = _product(s, "w")
            if s["bias"] is not None:
                z = z + s["bias"].float()
            y = _act(z, c["act"])
            if s["residual"] is not None:
                y = y + s["residual"].float()
            return dict(y=y.to(bf16), z=z.to(bf16)) if c["save"] else dict(y=y.to(bf16))
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_grad(s["z"].float(), c["act"])
        o = dict(dx=(dz @ s["w"].float()).to(bf16), dw=(dz.T @ s["x"].float()).to(bf16))
        if c["bias"]:
            o["db"] = dz.sum(0).to(bf16)
        return o
    if c["dir"] == "fwd":
        g, u = _product(s, "wg"), _product(s, "wu")
        h = (_act(g, c["act"]) * u).to(bf16)
        return dict(h=h, g=g.to(bf16), u=u.to(bf16)) if c["save"] else dict(h=h)
    dh, g, u, x = s["dh"].float(), s["g"].float(), s["u"].float(), s["x"].float()
    dg, du = dh * u * _act_grad(g, c["act"]), dh * _act(g, c["act"])
    dx = dg @ s["wg"].float() + du @ s["wu"].float()
    return dict(dx=dx.to(bf16), dwg=(dg.T @ x).to(bf16), dwu=(du.T @ x).to(bf16))


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits; gradients by differentiation of the definition."""
    F = torch.nn.functional
    d = {k: v.double() for k, v in _inputs(case, seed).items() if v is not None}
    n, k = case["n"], case["k"]
    fs = {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
          "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            var, mean = torch.var_mean(d["x"], 1, correction=0)
            y = F.layer_norm(d["x"], (k,), d["gamma"], d["beta"], EPS)
            return dict(y=y, mean=mean, rstd=torch.rsqrt(var + EPS))
        # mean and rstd are the forward pass's, rounded to 32 bits: closer to x's own than the outputs resolve
        leaf = [d[v].requires_grad_() for v in ("x", "gamma", "beta")]
        dx, dgamma, dbeta = torch.autograd.grad(F.layer_norm(leaf[0], (k,), leaf[1], leaf[2], EPS), leaf, d["dy"])
        return dict(dx=dx + d["dres"] if "dres" in d else dx, dgamma=dgamma, dbeta=dbeta)
    f = fs[case["act"]]

    def scaled(name):
        return d[name] * d["scale_" + name] if "scale_" + name in d else d[name]

    if case["op"] == "linear" and case["dir"] == "fwd":
        z = F.linear(scaled("x"), scaled("w"), d.get("bias"))
        o = dict(y=f(z) + d.get("residual", 0))
        return dict(o, z=z) if case["save"] else o
    if case["op"] == "linear":
        dz = d["dy"]
        if "z" in d:
            z = d["z"].requires_grad_()
            dz, = torch.autograd.grad(f(z), z, dz)
        o = dict(dx=torch.einsum("nm,mk->nk", dz, d["w"]), dw=torch.einsum("nm,nk->mk", dz, d["x"]))
        return dict(o, db=dz.sum(0)) if case["bias"] else o
    if case["dir"] == "fwd":
        x = scaled("x")
        g, u = F.linear(x, scaled("wg")), F.linear(x, scaled("wu"))
        return dict(h=f(g) * u, g=g, u=u) if case["save"] else dict(h=f(g) * u)
    g, u = d["g"].requires_grad_(), d["u"].requires_grad_()
    dg, du = torch.autograd.grad(f(g) * u, (g, u), d["dh"])
    return dict(dx=torch.einsum("nm,mk->nk", dg, d["wg"]) + torch.einsum("nm,mk->nk", du, d["wu"]),
                dwg=torch.einsum("nm,nk->mk", dg, d["x"]), dwu=torch.einsum("nm,nk->mk", du, d["x"]))
