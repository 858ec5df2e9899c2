"""A gated feed-forward sublayer from the library's calls: y = x + down(gated(norm(x))).

    python -m tensor_comm_gemm_gb300.ffn_layer --tokens 4096 --hidden 4096 --ffn 14336 --train
    python -m tensor_comm_gemm_gb300.ffn_layer --tokens 2048 --hidden 4096 --ffn 14336 --tp 4
    python -m tensor_comm_gemm_gb300.ffn_layer --tokens 1 --hidden 8192 --ffn 3584

With --tp 1 the down projection adds the residual in its epilogue, and --train
runs the backward pass through all three operators.  With more ranks each rank
holds a slice of the feed-forward width: every rank's gated projections run on
its own weights, and the row-parallel down projection is the library's
GEMM+AR over the ranks' slices.  Prints the time of a step and, with --check,
the largest error of each result against 64-bit arithmetic.
"""

import argparse

import torch

from . import tpoverlap as t

BF16 = torch.bfloat16
EPS = 1e-5


class FfnLayer:
    """Weights, saved activations and handles of one sublayer on the current device."""

    def __init__(self, hidden: int, ffn: int, tp: int = 1, max_tokens: int = 4096, seed: int = 0, train: bool = False):
        if ffn % tp or (train and tp != 1):
            raise ValueError("ffn must be a multiple of tp, and training runs with tp=1")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF16)

        self.hidden, self.ffn, self.tp, self.max_tokens = hidden, ffn, tp, max_tokens
        part = ffn // tp
        self.gamma = (1 + torch.randn(hidden, generator=gen, device="cuda") * 0.1).to(BF16)
        self.beta = normal(hidden, scale=0.1)
        self.wg = [normal(part, hidden, scale=hidden ** -0.5) for _ in range(tp)]
        self.wu = [normal(part, hidden, scale=hidden ** -0.5) for _ in range(tp)]
        self.wd = [normal(hidden, part, scale=ffn ** -0.5) for _ in range(tp)]
        need = [0]
        if train:
            need = [t.tpo_block_workspace(op, max_tokens, hidden, ffn)
                    for op in (t.TPO_OP_LAYER_NORM_BWD, t.TPO_OP_GATED_BWD)]
            need.append(t.tpo_block_workspace(t.TPO_OP_LINEAR_BWD, max_tokens, ffn, hidden))
        self.block = t.tpo_block_create(max(need))
        self.ctx = {}  # GEMM+AR contexts by token count

    def close(self):
        t.tpo_block_destroy(self.block)
        for c in self.ctx.values():
            t.tpo_ctx_destroy(c)

    def buffers(self, tokens: int, train: bool = False):
        """What a program keeps for batches of this many tokens."""
        def e(*shape, dtype=BF16):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        part = self.ffn // self.tp
        b = dict(norm=e(tokens, self.hidden), h=[e(tokens, part) for _ in range(self.tp)], y=e(tokens, self.hidden),
                 mean=e(tokens, dtype=torch.float32), rstd=e(tokens, dtype=torch.float32))
        if train:
            b.update(g=e(tokens, part), u=e(tokens, part), dh=e(tokens, part), dnorm=e(tokens, self.hidden),
                     dx=e(tokens, self.hidden), dwg=e(part, self.hidden), dwu=e(part, self.hidden),
                     dwd=e(self.hidden, part), dgamma=e(self.hidden), dbeta=e(self.hidden))
        return b

    def forward(self, x, b, train: bool = False):
        t.tpo_layer_norm(self.block, x, self.gamma, self.beta, b["norm"], mean=b["mean"], rstd=b["rstd"], eps=EPS)
        for r in range(self.tp):
            t.tpo_gated(self.block, b["norm"], self.wg[r], self.wu[r], b["h"][r], act=t.TPO_ACT_SILU,
                        g=b["g"] if train else None, u=b["u"] if train else None)
        if self.tp == 1:
            t.tpo_linear(self.block, b["h"][0], self.wd[0], b["y"], residual=x)
        else:
            n = x.shape[0]
            if n not in self.ctx:
                self.ctx[n] = t.tpo_ctx_create(self.tp, n, self.ffn, self.hidden, t.TPO_BF16)
            t.tpo_gemm_ar(self.ctx[n], b["h"], self.wd, b["y"], 1)
            b["y"].add_(x)
        return b["y"]

    def backward(self, x, dy, b):
        """Gradients of x and of every weight from dy, into the buffers."""
        t.tpo_linear_bwd(self.block, dy, b["h"][0], self.wd[0], dx=b["dh"], dw=b["dwd"])
        t.tpo_gated_bwd(self.block, b["dh"], b["g"], b["u"], b["norm"], self.wg[0], self.wu[0], dx=b["dnorm"],
                        dwg=b["dwg"], dwu=b["dwu"], act=t.TPO_ACT_SILU)
        # the residual branch's gradient joins inside the norm's backward pass
        t.tpo_layer_norm_bwd(self.block, b["dnorm"], x, self.gamma, b["mean"], b["rstd"], b["dx"],
                             dgamma=b["dgamma"], dbeta=b["dbeta"], dres=dy)
        return b["dx"]

    def status(self):
        for st in [t.tpo_block_sync_status(self.block)] + [t.tpo_sync_status(c) for c in self.ctx.values()]:
            if st:
                raise t.TpoError(st, t.tpo_last_error())


def reference(layer: FfnLayer, x, dy=None):
    """The sublayer in 64 bits, and its gradients by differentiation."""
    d = lambda ws: torch.cat([w.double() for w in ws])  # noqa: E731
    leaf = dict(x=x.double(), gamma=layer.gamma.double(), beta=layer.beta.double(), wg=d(layer.wg), wu=d(layer.wu),
                wd=torch.cat([w.double() for w in layer.wd], 1))
    for v in leaf.values():
        v.requires_grad_()
    f = torch.nn.functional
    norm = f.layer_norm(leaf["x"], (layer.hidden,), leaf["gamma"], leaf["beta"], EPS)
    h = f.silu(norm @ leaf["wg"].T) * (norm @ leaf["wu"].T)
    y = leaf["x"] + h @ leaf["wd"].T
    out = dict(y=y.detach())
    if dy is not None:
        for name, g in zip(leaf, torch.autograd.grad(y, list(leaf.values()), dy.double())):
            out["d" + name] = g
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, required=True)
    ap.add_argument("--hidden", type=int, required=True)
    ap.add_argument("--ffn", type=int, required=True)
    ap.add_argument("--tp", type=int, default=1, help="simulated ranks that share the feed-forward width")
    ap.add_argument("--train", action="store_true", help="forward and backward pass")
    ap.add_argument("--check", action="store_true", help="compare with 64-bit arithmetic")
    ap.add_argument("--calls", type=int, default=20)
    args = ap.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("ffn_layer needs a CUDA device")
    layer = FfnLayer(args.hidden, args.ffn, args.tp, args.tokens, train=args.train)
    try:
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        x = torch.randn(args.tokens, args.hidden, generator=gen, device="cuda").to(BF16)
        dy = torch.randn(args.tokens, args.hidden, generator=gen, device="cuda").to(BF16)
        b = layer.buffers(args.tokens, args.train)

        def step():
            layer.forward(x, b, args.train)
            if args.train:
                layer.backward(x, dy, b)

        for _ in range(3):
            step()
        layer.status()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(args.calls):
            step()
        end.record()
        layer.status()
        us = start.elapsed_time(end) * 1e3 / args.calls
        flops = 6.0 * args.tokens * args.hidden * args.ffn * (3 if args.train else 1)
        print("%d tokens, %d hidden, %d ffn, tp %d%s: %.1f us a step, %.1f TFLOP/s" % (
            args.tokens, args.hidden, args.ffn, args.tp, ", forward and backward" if args.train else "", us,
            flops / us * 1e-6))
        errors = {}
        if args.check:
            want = reference(layer, x, dy if args.train else None)
            got = dict(y=b["y"])
            if args.train:
                got.update(dx=b["dx"], dgamma=b["dgamma"], dbeta=b["dbeta"], dwg=b["dwg"], dwu=b["dwu"], dwd=b["dwd"])
            for name, v in got.items():
                errors[name] = float((v.double() - want[name]).norm() / want[name].norm())
            print("relative errors: " + ", ".join("%s %.2e" % e for e in errors.items()))
        return errors
    finally:
        layer.close()


if __name__ == "__main__":
    main()
