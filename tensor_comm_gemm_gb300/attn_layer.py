"""An attention sublayer from the library's calls: y = x + out(attention(rotary(qkv(norm(x))))).

    python -m tensor_comm_gemm_gb300.attn_layer --tokens 4096 --hidden 4096 --heads 32 --kv-heads 8 --train
    python -m tensor_comm_gemm_gb300.attn_layer --tokens 2048 --hidden 4096 --heads 32 --kv-heads 8 --tp 4 --sequences 5
    python -m tensor_comm_gemm_gb300.attn_layer --tokens 16 --hidden 4096 --heads 32 --kv-heads 8 --cache 8192

The tokens are --sequences packed sequences, each causal.  With --cache every
token is the next one of a sequence of its own: its key and value go into the
sequence's rows of a cache of that many rows, and it attends over them.  With
--tp 1 the output projection adds the residual in its epilogue, and --train runs
the backward pass through all operators.  With more ranks each rank holds a slice
of the heads, and the row-parallel output projection is the library's GEMM+AR
over the ranks' slices.  Prints the time of a step and, with --check, the relative
error of each result against 64-bit arithmetic: of the output and of attention's
alone, of the gradients, and of the rows that a step writes into a cache, whose
other rows must stay as they were.
"""

import argparse

import torch

from . import tpoverlap as t

BF16 = torch.bfloat16
EPS = 1e-5
BASE = 10000.0


class AttnLayer:
    """Weights, caches, saved activations and handles of one sublayer on the current device."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, dim: int = 128, tp: int = 1, max_tokens: int = 4096,
                 cache: int = 0, seed: int = 0, train: bool = False):
        if heads % tp or kv_heads % tp or (train and (tp != 1 or cache)):
            raise ValueError("heads and kv_heads must be multiples of tp, and training runs with tp=1 and no cache")
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF16)

        self.hidden, self.heads, self.kv, self.dim, self.tp = hidden, heads // tp, kv_heads // tp, dim, tp
        self.cache, width = cache, (self.heads + 2 * self.kv) * dim
        self.gamma = (1 + torch.randn(hidden, generator=gen, device="cuda") * 0.1).to(BF16)
        self.beta = normal(hidden, scale=0.1)
        self.wqkv = [normal(width, hidden, scale=hidden ** -0.5) for _ in range(tp)]
        self.wo = [normal(hidden, self.heads * dim, scale=(heads * dim) ** -0.5) for _ in range(tp)]
        self.table = t.tpo_rotary_table(dim, BASE).cuda()
        if cache:  # keys and values of max_tokens sequences
            self.k = [normal(max_tokens * cache, self.kv, dim, scale=1.0) for _ in range(tp)]
            self.v = [normal(max_tokens * cache, self.kv, dim, scale=1.0) for _ in range(tp)]
        need = [t.tpo_attention_workspace(max_tokens, max_tokens * max(cache, 1), self.heads, self.kv, dim)]
        if train:
            need.append(t.tpo_attention_bwd_workspace(max_tokens, max_tokens, heads, kv_heads, dim))
            need.append(t.tpo_block_workspace(t.TPO_OP_LAYER_NORM_BWD, max_tokens, hidden, 1))
            need += [t.tpo_block_workspace(t.TPO_OP_LINEAR_BWD, max_tokens, k, m)
                     for k, m in ((heads * dim, hidden), (hidden, width))]
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

        all_heads = self.heads + 2 * self.kv
        b = dict(norm=e(tokens, self.hidden), qkv=[e(tokens, all_heads, self.dim) for _ in range(self.tp)],
                 out=[e(tokens, self.heads, self.dim) for _ in range(self.tp)], y=e(tokens, self.hidden),
                 mean=e(tokens, dtype=torch.float32), rstd=e(tokens, dtype=torch.float32))
        if train:
            b.update(lse=e(tokens, self.heads, dtype=torch.float32), dout=e(tokens, self.heads, self.dim),
                     dqkv=e(tokens, all_heads, self.dim), dnorm=e(tokens, self.hidden), dx=e(tokens, self.hidden),
                     dwqkv=torch.empty_like(self.wqkv[0]), dwo=torch.empty_like(self.wo[0]), dgamma=e(self.hidden),
                     dbeta=e(self.hidden))
        return b

    def slices(self, qkv):
        return qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]

    def _project(self, x, b):
        t.tpo_layer_norm(self.block, x, self.gamma, self.beta, b["norm"], mean=b["mean"], rstd=b["rstd"], eps=EPS)
        for w, qkv in zip(self.wqkv, b["qkv"]):
            t.tpo_linear(self.block, b["norm"], w, qkv.view(len(x), -1))

    def _output(self, x, b):
        outs = [o.view(len(x), -1) for o in b["out"]]
        if self.tp == 1:
            t.tpo_linear(self.block, outs[0], self.wo[0], b["y"], residual=x)
        else:
            n, k = len(x), self.heads * self.dim * self.tp
            if n not in self.ctx:
                self.ctx[n] = t.tpo_ctx_create(self.tp, n, k, self.hidden, t.TPO_BF16)
            t.tpo_gemm_ar(self.ctx[n], outs, self.wo, b["y"], 1)
            b["y"].add_(x)
        return b["y"]

    def forward(self, x, pos, start, b, train: bool = False):
        """Packed sequences: rows [start[i], start[i + 1]) with positions pos."""
        self._project(x, b)
        for qkv, out in zip(b["qkv"], b["out"]):
            turned = qkv[:, :self.heads + self.kv]  # queries and keys, in place
            t.tpo_rotary(self.block, turned, self.table, turned, pos=pos)
            t.tpo_attention(self.block, *self.slices(qkv), out, q_start=start, lse=b["lse"] if train else None)
        return self._output(x, b)

    def decode(self, x, pos, where, b):
        """A token of each sequence, at position pos of its rows of the cache; where: start (one more than there are
        tokens), k_start, rows (of the tokens) and k_len (with them), int32."""
        self._project(x, b)
        for r, (qkv, out) in enumerate(zip(b["qkv"], b["out"])):
            q, k, v = self.slices(qkv)
            t.tpo_rotary(self.block, q, self.table, q, pos=pos)
            t.tpo_rotary(self.block, k, self.table, self.k[r], pos=pos, rows=where["rows"])
            t.tpo_rotary(self.block, v, None, self.v[r], rows=where["rows"])  # a copy
            t.tpo_attention(self.block, q, self.k[r], self.v[r], out, q_start=where["start"], k_start=where["k_start"],
                            k_len=where["k_len"])
        return self._output(x, b)

    def backward(self, x, dy, pos, start, b):
        """Gradients of x and of every weight from dy, into the buffers."""
        n = len(x)
        t.tpo_linear_bwd(self.block, dy, b["out"][0].view(n, -1), self.wo[0], dx=b["dout"].view(n, -1), dw=b["dwo"])
        t.tpo_attention_bwd(self.block, b["dout"], *self.slices(b["qkv"][0]), b["out"][0], b["lse"],
                            *self.slices(b["dqkv"]), q_start=start)
        turned = b["dqkv"][:, :self.heads + self.kv]
        t.tpo_rotary(self.block, turned, self.table, turned, pos=pos, inverse=True)
        t.tpo_linear_bwd(self.block, b["dqkv"].view(n, -1), b["norm"], self.wqkv[0], dx=b["dnorm"], dw=b["dwqkv"])
        # the residual branch's gradient joins inside the norm's backward pass
        t.tpo_layer_norm_bwd(self.block, b["dnorm"], x, self.gamma, b["mean"], b["rstd"], b["dx"], dgamma=b["dgamma"],
                             dbeta=b["dbeta"], dres=dy)
        return b["dx"]

    def status(self):
        for st in [t.tpo_block_sync_status(self.block)] + [t.tpo_sync_status(c) for c in self.ctx.values()]:
            if st:
                raise t.TpoError(st, t.tpo_last_error())


def _turn(x, pos):
    """Rotary positions of [n, heads, dim] in 64 bits."""
    half = x.shape[2] // 2
    f = BASE ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    a = (pos.double()[:, None] * f)[:, None]
    lo, hi = x[..., :half], x[..., half:]
    return torch.cat([lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()], 2)


def reference(layer: AttnLayer, x, pos, lens, dy=None, old=None):
    """The sublayer in 64 bits (y, and out of the attention alone), and its gradients by differentiation.  lens: the
    packed sequences' lengths, or with `old` (caches before the step, of each rank) the keys of each token's sequence, its
    own the last of them; k and v are then the tokens' rows of the caches."""
    leaf = dict(x=x.double(), gamma=layer.gamma.double(), beta=layer.beta.double(),
                wqkv=torch.cat([w.double() for w in layer.wqkv]), wo=torch.cat([w.double() for w in layer.wo], 1))
    for v in leaf.values():
        v.requires_grad_()
    norm = torch.nn.functional.layer_norm(leaf["x"], (layer.hidden,), leaf["gamma"], leaf["beta"], EPS)
    outs, keys, values = [], [], []
    for r, w in enumerate(leaf["wqkv"].chunk(layer.tp)):
        q, k, v = layer.slices((norm @ w.T).view(len(x), -1, layer.dim))
        q, k = _turn(q, pos), _turn(k, pos)
        at, rows = 0, []
        for i, n in enumerate(lens):
            if old is None:
                qs, ks, vs = q[at:at + n], k[at:at + n], v[at:at + n]
                at += n
            else:
                past = slice(i * layer.cache, i * layer.cache + n - 1)
                qs = q[i:i + 1]
                ks, vs = (torch.cat([c[past].double(), y[i:i + 1]]) for c, y in ((old[0][r], k), (old[1][r], v)))
            ks, vs = (y.repeat_interleave(layer.heads // layer.kv, 1) for y in (ks, vs))
            z = torch.einsum("qhd,khd->hqk", qs, ks) * layer.dim ** -0.5
            hidden = torch.ones(z.shape[1:], dtype=torch.bool, device=z.device).triu(1 + z.shape[2] - z.shape[1])
            p = z.masked_fill(hidden, float("-inf")).softmax(2)
            rows.append(torch.einsum("hqk,khd->qhd", p, vs))
        outs.append(torch.cat(rows).flatten(1))
        keys.append(k)
        values.append(v)
    y = leaf["x"] + torch.cat(outs, 1) @ leaf["wo"].T
    out = dict(y=y.detach(), out=torch.cat(outs, 1).detach())
    if old is not None:
        out.update(k=torch.cat(keys, 1).detach(), v=torch.cat(values, 1).detach())
    if dy is not None:
        for name, g in zip(leaf, torch.autograd.grad(y, list(leaf.values()), dy.double())):
            out["d" + name] = g
    return out


def compare(layer: AttnLayer, b, want, rows=None, old=None):
    """The error of each of reference()'s results relative to its own size: y alone would hide attention's behind the
    residual.  With caches (`old`: before the step) also how many elements behind the step's `rows` have changed."""
    got, errors = dict(b, out=torch.cat([o.flatten(1) for o in b["out"]], 1)), {}
    if old is not None:
        rows = rows.long()
        for name, now, before in (("k", layer.k, old[0]), ("v", layer.v, old[1])):
            got[name] = torch.cat([c[rows] for c in now], 1)
            changed = [(c.view(torch.int16) != o.view(torch.int16)).index_fill_(0, rows, False) for c, o in zip(now, before)]
            errors["other rows of " + name] = float(sum(c.sum() for c in changed))
    for name in want:
        errors[name] = float((got[name].double() - want[name]).norm() / want[name].norm())
    return errors


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, required=True)
    ap.add_argument("--hidden", type=int, required=True)
    ap.add_argument("--heads", type=int, required=True)
    ap.add_argument("--kv-heads", type=int, required=True)
    ap.add_argument("--dim", type=int, default=128)
    ap.add_argument("--sequences", type=int, default=1, help="packed sequences of about equal lengths")
    ap.add_argument("--cache", type=int, default=0,
                    help="each token is the next of a sequence with a cache of so many rows")
    ap.add_argument("--tp", type=int, default=1, help="simulated ranks that share the heads")
    ap.add_argument("--train", action="store_true", help="forward and backward pass")
    ap.add_argument("--check", action="store_true", help="compare with 64-bit arithmetic")
    ap.add_argument("--calls", type=int, default=20)
    args = ap.parse_args(argv)
    if not torch.cuda.is_available():
        raise SystemExit("attn_layer needs a CUDA device")
    layer = AttnLayer(args.hidden, args.heads, args.kv_heads, args.dim, args.tp, args.tokens, args.cache,
                      train=args.train)
    try:
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        x = torch.randn(args.tokens, args.hidden, generator=gen, device="cuda").to(BF16)
        dy = torch.randn(args.tokens, args.hidden, generator=gen, device="cuda").to(BF16)
        b = layer.buffers(args.tokens, args.train)

        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device="cuda")

        if args.cache:  # full but for a few rows, a different number in each
            lens = [max(1, args.cache - 5 * i % (args.cache // 2 + 1)) for i in range(args.tokens)]
            pos = ints([n - 1 for n in lens])
            where = dict(start=ints(range(args.tokens + 1)), k_len=ints(lens),
                         k_start=ints([i * args.cache for i in range(args.tokens)]),
                         rows=ints([i * args.cache + n - 1 for i, n in enumerate(lens)]))
            pairs = sum(lens)
        else:
            cuts = [args.tokens * i // args.sequences for i in range(args.sequences + 1)]
            lens = [e - s for s, e in zip(cuts, cuts[1:])]
            pos, start = ints([i for n in lens for i in range(n)]), ints(cuts)
            pairs = sum(n * (n + 1) // 2 for n in lens)
        old = ([k.clone() for k in layer.k], [v.clone() for v in layer.v]) if args.cache and args.check else None

        def step():
            if args.cache:
                layer.decode(x, pos, where, b)
                return
            layer.forward(x, pos, start, b, args.train)
            if args.train:
                layer.backward(x, dy, pos, start, b)

        for _ in range(3):
            step()
        layer.status()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(args.calls):
            step()
        end.record()
        layer.status()
        us = begin.elapsed_time(end) * 1e3 / args.calls
        linear = 2.0 * args.tokens * args.hidden * args.dim * (2 * args.heads + 2 * args.kv_heads)
        flops = linear * (3 if args.train else 1) + 4.0 * pairs * args.heads * args.dim * (3.5 if args.train else 1)
        print("%d tokens, %d hidden, %d heads of %d over %d, %s, tp %d%s: %.1f us a step, %.1f TFLOP/s" % (
            args.tokens, args.hidden, args.heads, args.dim, args.kv_heads,
            "a cache of %d" % args.cache if args.cache else "%d sequences" % args.sequences, args.tp,
            ", forward and backward" if args.train else "", us, flops / us * 1e-6))
        errors = {}
        if args.check:
            want = reference(layer, x, pos, lens, dy if args.train else None, old)
            errors = compare(layer, b, want, where["rows"] if args.cache else None, old)
            print("relative errors: " + ", ".join("%s %.2e" % e for e in errors.items()))
        return errors
    finally:
        layer.close()


if __name__ == "__main__":
    main()
