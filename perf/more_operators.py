"""Cases of the attention sublayer's operators: rotary positions, and attention
with grouped heads over packed sequences, forward, backward and over a cache.

A case names an operator ("op"), a direction ("dir") and sizes:

  rotary     x [n, heads, dim]: the first `rot` elements of each head turn by the
             token's position; the backward pass turns the other way;
  attention  q [n, heads, dim] over k and v [nk, kv_heads, dim], sequence by
             sequence, query i of nq seeing the keys up to i + nk - nq (causal)
             or all of its sequence, and the backward pass.

"lens" holds the sequences' numbers of queries, "klens" those of keys (empty:
the same), as text.  "cache" > 0: keys and values lie in a cache of that many
rows per sequence.  "fused": q, k and v are slices of one projection's output.
Heads are those of one rank of a tensor-parallel layer.
"""

import math
import weakref

import torch

own = False

LARGEST_FLOPS = 2.5 * 4 * 128 * 32 * 2 * (4096 * 4097 // 2)
LARGEST_BYTES = 1.0e9
LARGEST_SCORES = 2.2e9  # of the padded plain form: heads x sequences x longest x longest


def listed():
    return [
        # Queries and keys of one generated token, deep in a context.
        dict(name="rotary_token", op="rotary", dir="fwd", dtype="bf16", n=1, heads=40, dim=128, rot=128,
             layout="half", scaling="none", start=9000, pad=8),
        # Those of a long prompt's last part, the context four times the trained one.
        dict(name="rotary_prompt", op="rotary", dir="fwd", dtype="bf16", n=8192, heads=72, dim=128, rot=128,
             layout="half", scaling="parts", start=122880, pad=8),
        # Gradient of a full-precision layer that turns part of each head, pairs side by side; odd sizes.
        dict(name="rotary_grad", op="rotary", dir="bwd", dtype="f32", n=5003, heads=9, dim=80, rot=32,
             layout="interleaved", scaling="linear", start=0, pad=0),
        # A short prompt on one rank of eight: latency only.
        dict(name="prompt_short", op="attention", dir="fwd", lens="37", klens="", heads=8, kv_heads=1, dim=128,
             causal=True, save=False, cache=0, fused=True),
        # A long prompt of a layer 4096 wide.
        dict(name="prompt_long", op="attention", dir="fwd", lens="8192", klens="", heads=32, kv_heads=8, dim=128,
             causal=True, save=False, cache=0, fused=True),
        # Packed training sequences of different lengths on one rank of eight.
        dict(name="prompt_packed", op="attention", dir="fwd", lens="2311,17,1024,640,1,1999,333,128,901,257,45,536",
             klens="", heads=8, kv_heads=1, dim=128, causal=True, save=True, cache=0, fused=True),
        # Both directions of an encoder with small heads.
        dict(name="prompt_both_ways", op="attention", dir="fwd", lens="1024,777,513,1024,60,1024,999,1024", klens="",
             heads=16, kv_heads=16, dim=64, causal=False, save=True, cache=0, fused=False),
        # The next part of a prompt whose earlier tokens lie in the cache.
        dict(name="prompt_part", op="attention", dir="fwd", lens="512", klens="25088", heads=8, kv_heads=1, dim=128,
             causal=True, save=False, cache=32768, fused=False),
        # Training's backward pass of a layer 4096 wide; the largest case.
        dict(name="backward", op="attention", dir="bwd", lens="4096,4096", klens="", heads=32, kv_heads=8, dim=128,
             causal=True, save=True, cache=0, fused=True),
        # The same for odd lengths, heads and head size.
        dict(name="backward_odd", op="attention", dir="bwd", lens="1333,75,2047,1,410", klens="", heads=9, kv_heads=3,
             dim=80, causal=True, save=True, cache=0, fused=False),
        # One token of one long sequence on one rank of eight.
        dict(name="token_long", op="attention", dir="fwd", lens="1", klens="32768", heads=8, kv_heads=1, dim=128,
             causal=True, save=False, cache=40960, fused=False),
        # One token of each of 64 sequences.
        dict(name="tokens_batch", op="attention", dir="fwd", lens=",".join(["1"] * 64),
             klens=",".join(str(17 + 8175 * ((i * 37) % 64) // 63) for i in range(64)), heads=32, kv_heads=8, dim=128,
             causal=True, save=False, cache=8192, fused=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    while True:
        if rng.random() < 0.25:
            dim = 8 * rng.choice((4, 6, 8, 10, 12, 16, 16))
            c = dict(op="rotary", dir=rng.choice(("fwd", "fwd", "bwd")), dtype=rng.choice(("bf16", "bf16", "f32")),
                     n=_log(rng, 1, 8192), heads=_log(rng, 1, 72), dim=dim,
                     rot=rng.choice((dim, dim, dim // 2, dim // 4)) // 2 * 2, layout=rng.choice(("half", "interleaved")),
                     scaling=rng.choice(("none", "linear", "parts")), start=rng.choice((0, 1, 4095, 100000, 1000000)),
                     pad=rng.choice((0, 0, 8)))
            if work(c)["bytes"] <= LARGEST_BYTES:
                return c
            continue
        kind = rng.choice(("prompt", "prompt", "backward", "backward", "tokens", "part"))
        kv = rng.choice((1, 1, 2, 3, 4, 8))
        c = dict(op="attention", dir="bwd" if kind == "backward" else "fwd", heads=kv * rng.choice((1, 2, 3, 4, 5, 8, 8)),
                 kv_heads=kv, dim=8 * rng.choice((4, 5, 8, 8, 10, 12, 16, 16, 16)), causal=rng.random() < 0.75)
        if kind == "tokens":
            count, longest, few = _log(rng, 1, 96), _log(rng, 16, 32768), rng.choice((1, 1, 1, 2, 4))
            klens = [max(few, rng.randint(1, longest)) for _ in range(count)]
            lens, c["cache"] = [few] * count, max(klens) + rng.randint(0, 64)
        elif kind == "part":
            lens = [_log(rng, 8, 1024) for _ in range(_log(rng, 1, 4))]
            klens = [v + _log(rng, 1, 16384) for v in lens]
            c["cache"] = max(klens) + rng.randint(0, 64)
        else:
            longest = _log(rng, 2, 8192)
            lens = [max(1, rng.randint(longest // 8, longest)) for _ in range(_log(rng, 1, 16))]
            klens, c["cache"] = [], 0
        c.update(lens=",".join(map(str, lens)), klens=",".join(map(str, klens)), fused=not klens and rng.random() < 0.5,
                 save=kind == "backward" or rng.random() < 0.3)
        w = work(c)
        scores = c["heads"] * len(lens) * max(lens) * max(klens or lens)
        if w["flops"] <= LARGEST_FLOPS and w["bytes"] <= LARGEST_BYTES and scores <= LARGEST_SCORES:
            return c


def _lens(case):
    q = [int(v) for v in case["lens"].split(",")]
    return q, [int(v) for v in case["klens"].split(",")] if case["klens"] else q


def _pairs(case):
    """(query, key) pairs that see each other."""
    total = 0
    for nq, nk in zip(*_lens(case)):
        if not case["causal"]:
            total += nq * nk
            continue
        first = nk - nq + 1  # keys that query 0 sees
        skip = max(0, -first)
        total += (nq - skip) * (first + skip + nk) // 2 if skip < nq else 0
    return total


def work(case):
    if case["op"] == "rotary":
        e = 2 if case["dtype"] == "bf16" else 4
        size = case["n"] * case["heads"] * case["dim"]
        return {"bytes": 2 * size * e + 4 * case["n"] + 4 * case["rot"], "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    q, k = _lens(case)
    nq = sum(q) * case["heads"] * case["dim"]
    nk = sum(k) * case["kv_heads"] * case["dim"]
    lse = 4 * sum(q) * case["heads"]
    flops = 4 * case["dim"] * case["heads"] * _pairs(case)
    if case["dir"] == "bwd":  # reads q, out, dout, k, v and lse, writes dq, dk and dv
        return {"bytes": 8 * nq + 8 * nk + lse, "flops": 5 * flops // 2}
    return {"bytes": 4 * nq + 4 * nk + (lse if case["save"] else 0), "flops": flops}


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE, FACTOR, LOW, HIGH, ORIGINAL = 500000.0, 4.0, 1.0, 4.0, 32768


def _angles_per_position(case):
    """The `rot` / 2 frequencies in 64 bits."""
    i = torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / case["rot"])
    if case["scaling"] == "linear":
        return f / FACTOR
    if case["scaling"] == "parts":  # turns within the trained context: many stay, few stretch, a blend between
        turns = ORIGINAL * f / (2 * math.pi)
        keep = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        return f * (keep + (1 - keep) / FACTOR)
    return f


def _inputs(case, seed):
    """The tensors of one case, from its seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)

    if case["op"] == "rotary":
        n, heads, dim = case["n"], case["heads"], case["dim"]
        wide = normal(n, heads + case["pad"], dim, dtype=_TYPES[case["dtype"]])  # the values' heads follow
        pos = torch.arange(case["start"], case["start"] + n, device="cuda", dtype=torch.int32)
        return dict(x=wide[:, :heads], pos=pos, freq=_angles_per_position(case).cuda())
    q_lens, k_lens = _lens(case)
    n, heads, kv, dim = sum(q_lens), case["heads"], case["kv_heads"], case["dim"]
    t = {}
    # a few channels of the keys are larger than the rest, as they are behind a trained projection
    channel = 0.8 + 2.0 * (torch.rand(kv, dim, generator=gen, device="cuda") < 0.04).float()
    if case["fused"]:
        qkv = normal(n, heads + 2 * kv, dim)
        qkv[:, heads:heads + kv] = (qkv[:, heads:heads + kv].float() * channel).to(torch.bfloat16)
        t["q"], t["k"], t["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        rows = case["cache"] * len(k_lens) if case["cache"] else sum(k_lens)
        t["q"] = normal(n, heads, dim)
        t["k"] = (torch.randn(rows, kv, dim, generator=gen, device="cuda") * channel).to(torch.bfloat16)
        t["v"] = normal(rows, kv, dim)
    if case["dir"] == "bwd":
        t["dout"] = normal(n, heads, dim)
    return t


class _Block:
    """The operators' handle and its workspace, given back with the state."""

    def __init__(self, binding, need):
        self.handle = binding.tpo_block_create(need)
        weakref.finalize(self, binding.tpo_block_destroy, self.handle)


def _cumulative(lens):
    at = [0]
    for v in lens:
        at.append(at[-1] + v)
    return at


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=dict(case))
    if case["op"] == "attention":
        # where each sequence's rows begin, and for the padded form every row's place
        q_lens, k_lens = _lens(case)
        q_at = _cumulative(q_lens)
        k_at = [i * case["cache"] for i in range(len(k_lens))] if case["cache"] else _cumulative(k_lens)
        lq, lk = torch.tensor(q_lens, device="cuda"), torch.tensor(k_lens, device="cuda")
        s["q_start"] = torch.tensor(q_at, device="cuda", dtype=torch.int32)
        s["k_start"] = torch.tensor(k_at, device="cuda", dtype=torch.int32)
        s["k_len"] = lk.to(torch.int32)
        iq, ik = torch.arange(max(q_lens), device="cuda"), torch.arange(max(k_lens), device="cuda")
        rq, rk = iq[None] < lq[:, None], ik[None] < lk[:, None]
        s["rows_q"] = torch.where(rq, iq[None] + s["q_start"][:len(q_lens), None], 0)
        s["rows_k"] = torch.where(rk, ik[None] + s["k_start"][:len(k_lens), None], 0)
        s["flat_q"], s["flat_k"] = rq.flatten().nonzero().flatten(), rk.flatten().nonzero().flatten()
        last = iq[None, :, None] + (lk - lq)[:, None, None] if case["causal"] else lk[:, None, None] + 0 * iq[None, :, None]
        s["sees"] = (ik[None, None] <= last) & rk[:, None] & rq[:, :, None]  # [sequences, queries, keys]
        if case["dir"] == "bwd":
            o = _attend(s)
            s["out"], s["lse"] = o["out"], o["lse"]
    if not own:
        return s
    from tensor_comm_gemm_gb300 import tpoverlap as t

    s["t"] = t
    if case["op"] == "rotary":
        scaling = {"none": t.TPO_ROTARY_UNSCALED, "linear": t.TPO_ROTARY_LINEAR, "parts": t.TPO_ROTARY_BY_PARTS}
        s["table"] = t.tpo_rotary_table(case["rot"], BASE, scaling[case["scaling"]], FACTOR, LOW, HIGH, ORIGINAL).cuda()
        s["layout"] = {"half": t.TPO_ROTARY_HALVES, "interleaved": t.TPO_ROTARY_PAIRS}[case["layout"]]
        s["block"] = _Block(t, 0)
        s["o"] = dict(y=torch.empty(case["n"], case["heads"], case["dim"], dtype=s["x"].dtype, device="cuda"))
        return s
    sizes = (s["q"].shape[0], s["k"].shape[0], case["heads"], case["kv_heads"], case["dim"])
    if case["dir"] == "fwd":
        s["block"] = _Block(t, t.tpo_attention_workspace(*sizes))
        s["o"] = dict(out=torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda"))
        if case["save"]:
            s["o"]["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
    else:
        s["block"] = _Block(t, t.tpo_attention_bwd_workspace(*sizes))
        s["o"] = {"d" + v: torch.empty(s[v].shape, dtype=s[v].dtype, device="cuda") for v in "qkv"}
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    t, c, o = s["t"], s["case"], s["o"]
    if c["op"] == "rotary":
        t.tpo_rotary(s["block"].handle, s["x"], s["table"], o["y"], pos=s["pos"], layout=s["layout"],
                     inverse=c["dir"] == "bwd")
        return o
    where = dict(q_start=s["q_start"], causal=c["causal"])
    if c["klens"]:
        where.update(k_start=s["k_start"], k_len=s["k_len"])
    if c["dir"] == "fwd":
        t.tpo_attention(s["block"].handle, s["q"], s["k"], s["v"], o["out"], lse=o.get("lse"), **where)
    else:
        t.tpo_attention_bwd(s["block"].handle, s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], o["dq"], o["dk"],
                            o["dv"], **where)
    return o


def _run_plain(s):
    c = s["case"]
    if c["op"] == "rotary":
        rot = c["rot"]
        turn = s["pos"].double()[:, None] * s["freq"]
        cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
        if c["dir"] == "bwd":
            sin = -sin
        x = s["x"].float()
        y = x.clone()
        if c["layout"] == "half":
            a, b = slice(0, rot // 2), slice(rot // 2, rot)
        else:
            a, b = slice(0, rot, 2), slice(1, rot, 2)
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., a] * sin + x[..., b] * cos
        return dict(y=y.to(s["x"].dtype))
    if c["dir"] == "fwd":
        return _attend(s)
    q, k, v, p = _weights(s, s["lse"])
    dout = _groups(s, s["dout"][s["rows_q"]].float())
    delta = _groups(s, (s["dout"].float() * s["out"].float()).sum(2, keepdim=True)[s["rows_q"]])
    dp = dout @ v.transpose(-1, -2)
    ds = dp.sub_(delta).mul_(p).mul_(c["dim"] ** -0.5)
    dq, dk, dv = ds @ k, (ds.transpose(-1, -2) @ q).sum(2), (p.transpose(-1, -2) @ dout).sum(2)
    bf16 = torch.bfloat16
    dq = dq.permute(0, 3, 1, 2, 4).flatten(2, 3).flatten(0, 1)[s["flat_q"]]
    dk, dv = (g.transpose(1, 2).flatten(0, 1)[s["flat_k"]] for g in (dk, dv))
    return dict(dq=dq.to(bf16), dk=dk.to(bf16), dv=dv.to(bf16))


def _groups(s, x):
    """[sequences, rows, heads, e] -> [sequences, key heads, heads of a group, rows, e]."""
    return x.unflatten(2, (s["case"]["kv_heads"], -1)).permute(0, 2, 3, 1, 4)


def _weights(s, lse=None):
    """q, k and v by sequence and head, and the weights: not yet divided by their sums, or with them known."""
    q = _groups(s, s["q"][s["rows_q"]].float())
    k, v = (_groups(s, s[x][s["rows_k"]].float()) for x in "kv")
    z = (q @ k.transpose(-1, -2)).mul_(s["case"]["dim"] ** -0.5).masked_fill_(~s["sees"][:, None, None], -math.inf)
    if lse is not None:
        known = _groups(s, lse[s["rows_q"]][..., None])
        return q, k, v, z.sub_(known.masked_fill(known == -math.inf, 0.0)).exp_()
    top = z.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0.0)
    return z.sub_(top).exp_(), v, top


def _attend(s):
    p, v, top = _weights(s)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.masked_fill(total == 0, 1.0)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3).flatten(0, 1)[s["flat_q"]].to(torch.bfloat16)
    if not s["case"]["save"]:
        return dict(out=out)
    lse = (top + total.log()).permute(0, 3, 1, 2, 4).flatten(2, 4).flatten(0, 1)[s["flat_q"]]
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The operators' definitions in 64 bits, sequence by sequence; gradients by differentiation of the definition."""
    t = _inputs(case, seed)
    if case["op"] == "rotary":
        rot, x = case["rot"], t["x"].double()
        pairs = x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else \
            x[..., :rot].unflatten(-1, (-1, 2))
        angle = t["pos"].double().outer(t["freq"])
        unit = torch.polar(torch.ones_like(angle), -angle if case["dir"] == "bwd" else angle)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit[:, None])
        turned = pairs.transpose(-1, -2) if case["layout"] == "half" else pairs
        return dict(y=torch.cat([turned.flatten(-2), x[..., rot:]], -1))
    group, scale = case["heads"] // case["kv_heads"], 1.0 / math.sqrt(case["dim"])
    made = {}
    q_at = k_at = 0
    for nq, nk in zip(*_lens(case)):
        for h in range(case["kv_heads"]):
            q = t["q"][q_at:q_at + nq, h * group:(h + 1) * group].double()
            k, v = (t[x][k_at:k_at + nk, h].double() for x in "kv")
            if case["dir"] == "bwd":
                for leaf in (q, k, v):
                    leaf.requires_grad_()
            z = torch.einsum("qgd,kd->gqk", q, k) * scale
            if case["causal"]:
                z = z.masked_fill(torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1), -math.inf)
            out = torch.einsum("gqk,kd->qgd", torch.softmax(z, -1), v)
            if case["dir"] == "bwd":
                dout = t["dout"][q_at:q_at + nq, h * group:(h + 1) * group].double()
                parts = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(out, (q, k, v), dout)))
                parts["dk"], parts["dv"] = parts["dk"][:, None], parts["dv"][:, None]
            else:
                parts = dict(out=out, lse=torch.logsumexp(z, -1).T) if case["save"] else dict(out=out)
            for name, value in parts.items():
                made.setdefault(name, []).append(value)
        q_at, k_at = q_at + nq, k_at + (case["cache"] or nk)
    kv, count = case["kv_heads"], len(_lens(case)[0])
    return {name: torch.cat([torch.cat(parts[i * kv:(i + 1) * kv], 1) for i in range(count)])
            for name, parts in made.items()}
