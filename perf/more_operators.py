"""What a training step runs around the blocks of a tensor-parallel stack, as cases to time.

Three operators, each with its backward pass where it has one:

* ``norm``: the end of one block and the start of the next in one pass: out =
  alpha x + gate * rmsnorm(y), a = rmsnorm(out); ``norm backward`` gives the gradients
  of the residual stream, the block's output, the gate and both weights;
* ``clip``: the norm of all gradients together, and the gradients scaled to at most
  a given norm;
* ``embed``: rows of a table whose vocabulary is split over ranks, scaled;
  ``embed backward`` gives the tables' gradients.

With ``own`` false, ``run`` computes them in elementary torch operations in 32 bits
(long sums in 64); with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a decoding request between two blocks: one launch, latency
        dict(name="norm one token", op="norm", T=1, H=8192, pad=0, x="bf16", y="bf16", a="bf16", param="bf16",
             use_y=True, post=True, groups=0, alpha=1.0, offset=0.0),
        # a decode step of 64 tokens: the all-reduce's fp32 output joins an fp32 stream,
        # the next products read bfloat16
        dict(name="norm decode", op="norm", T=64, H=4096, pad=0, x="f32", y="f32", a="bf16", param="f32",
             use_y=True, post=True, groups=1, alpha=1.0, offset=0.0),
        # a training or prefill step's tokens, everything in bfloat16, weights around 1, a scaled residual
        dict(name="norm training", op="norm", T=16384, H=8192, pad=0, x="bf16", y="bf16", a="bf16", param="bf16",
             use_y=True, post=True, groups=1, alpha=0.9375, offset=1.0),
        # its backward pass
        dict(name="norm backward training", op="norm backward", T=16384, H=8192, pad=0, x="bf16", y="bf16", a="bf16",
             param="bf16", use_y=True, post=True, groups=1, alpha=0.9375, offset=1.0),
        # backward on 2048 tokens of an fp32 stream with the reduced fp32 outputs, learned gates
        dict(name="norm backward f32", op="norm backward", T=2048, H=4096, pad=0, x="f32", y="f32", a="f32",
             param="f32", use_y=True, post=True, groups=1, alpha=1.0, offset=0.0),
        # a ragged batch of three sequences with a gate each, odd width, rows inside wider ones, backward
        dict(name="norm backward ragged", op="norm backward", T=3 * 347, H=1999, pad=7, x="f32", y="f16", a="f16",
             param="f32", use_y=True, post=False, groups=3, alpha=0.5, offset=0.0),
        # the gradients of a small stack's norm weights and gates: latency
        dict(name="clip small", op="clip", tensors=24, lo=4096, hi=4096, types="f32", max_norm=1.0, size=0.01),
        # the weight gradients of 8 layers split over 4 ranks (hidden 4096, ffn 16384), fp32
        dict(name="clip stack", op="clip", tensors=64, lo=4096 * 4096, hi=4096 * 4096, types="f32", max_norm=1.0,
             size=0.01),
        # many gradients of different types and odd lengths, below the limit
        dict(name="clip mixed", op="clip", tensors=331, lo=1, hi=1 << 20, types="f32 bf16 f16", max_norm=1000.0,
             size=0.01),
        # a decode step of 64 tokens: every one of 8 ranks' partials for the all-reduce
        dict(name="embed decode", op="embed", P=8, V=4096, T=64, H=4096, table="bf16", out="bf16", scale=64.0,
             first=0),
        # a prefill of 16384 tokens on a table that one GPU holds whole
        dict(name="embed prefill", op="embed", P=1, V=131072, T=16384, H=8192, table="bf16", out="bf16", scale=1.0,
             first=0),
        # the backward pass of a training step: tokens as frequent as words are, fp32 gradients
        # of the tables of 4 ranks
        dict(name="embed backward training", op="embed backward", P=4, V=16384, T=16384, H=4096, table="f32",
             out="f32", scale=64.0, first=0),
    ]


def _size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["norm", "norm backward", "clip", "embed", "embed backward"])
    if op.startswith("norm"):
        while True:
            half = rng.choice(["bf16", "bf16", "f16"])
            groups = rng.choice([0, 1, 1, 2, 5])
            T, H = _size(rng, 1, 16384), _size(rng, 64, 16384)
            if rng.random() < 0.6:
                H = -(-H // 64) * 64
            if groups > 1:
                T = -(-T // groups) * groups
            use_y = rng.random() < 0.85
            c = dict(op=op, T=T, H=H, pad=rng.choice([0, 0, 0, 8, 3]), x=rng.choice([half, "f32"]),
                     y=rng.choice([half, "f32"]), a=rng.choice([half, half, "f32"]), param=rng.choice(["f32", half]),
                     use_y=use_y, post=use_y and rng.random() < 0.6, groups=groups if use_y else 0,
                     alpha=rng.choice([1.0, 1.0, 0.5, 2.25]) if use_y else 1.0, offset=rng.choice([0.0, 1.0]))
            if T * H <= 1 << 26:
                return c
    if op == "clip":
        while True:
            lo = _size(rng, 1, 1 << 20)
            hi = min(1 << 26, lo * rng.choice([1, 7, 300]))
            c = dict(op=op, tensors=_size(rng, 1, 600), lo=lo, hi=hi,
                     types=rng.choice(["f32", "bf16", "f32 bf16", "f32 bf16 f16"]),
                     max_norm=rng.choice([1.0, 0.5, 1e4]), size=rng.choice([1e-3, 0.01, 1.0]))
            if c["tensors"] * hi <= 1 << 28:
                return c
    while True:
        t = rng.choice(["f32", "bf16", "bf16", "f16"])
        P = rng.choice([1, 1, 2, 4, 8])
        V, T, H = _size(rng, 32, 131072) // P + 1, _size(rng, 1, 32768), _size(rng, 64, 8192)
        if rng.random() < 0.6:
            H = -(-H // 64) * 64
        c = dict(op=op, P=P, V=V, T=T, H=H, table=t, out=rng.choice([t, "f32", "bf16"]) if t != "f16" else t,
                 scale=rng.choice([1.0, math.sqrt(H)]), first=rng.choice([0, 0, V]))
        if P * V * H <= 1 << 28 and (P if op == "embed" else 1) * T * H <= 1 << 26:
            return c


# ---- inputs ----------------------------------------------------------------------------------------------


def _clip_sizes(c):
    """The tensors' lengths and types: part of the case, the same for every seed."""
    rng = random.Random("%(tensors)d %(lo)d %(hi)d %(types)s" % c)
    types = c["types"].split()
    return [(_size(rng, c["lo"], c["hi"]), rng.choice(types)) for _ in range(c["tensors"])]


def _flat_views(c, dtypes, dev):
    """The clipped gradients as an optimizer keeps them: one buffer per type (zeros between the
    tensors), and a view of it for every tensor."""
    at, views = dict.fromkeys(DTYPES, 0), []
    for n, t in _clip_sizes(c):
        views.append((t, at[t], n))
        at[t] += -(-n // 64) * 64
    flat = {t: torch.zeros(n, dtype=dtypes[t], device=dev) for t, n in at.items() if n}
    return flat, [flat[t][lo:lo + n] for t, lo, n in views]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    c = dict(case)
    if c["op"].startswith("norm"):
        T, H, w = c["T"], c["H"], c["H"] + c["pad"]

        def matrix(dtype, size):
            return (size * normal(T, w)).to(DTYPES[dtype])[:, :H]

        def empty(dtype):
            return torch.empty(T, w, dtype=DTYPES[dtype], device=dev)[:, :H]

        channels = torch.exp(0.5 * normal(1, w))  # channels of a stream are of different size
        x = (channels * normal(T, w)).to(DTYPES[c["x"]])[:, :H]
        y = matrix(c["y"], 0.5) if c["use_y"] else None
        p = DTYPES[c["param"]]
        c["w_pre"] = (1.0 - c["offset"] + 0.2 * normal(H)).to(p)
        c["w_post"] = (1.0 - c["offset"] + 0.2 * normal(H)).to(p) if c["post"] else None
        c["gate"] = (0.5 + 0.3 * normal(c["groups"], H)).to(p) if c["groups"] else None
        c["x_t"], c["y_t"] = x, y
        if c["op"] == "norm":
            c["out_t"] = empty(c["x"]) if c["use_y"] else None
            c["a_t"] = empty(c["a"])
        else:
            # what arrives from the next block and along the residual stream
            c["dout_t"], c["da_t"] = matrix(c["x"], 0.01), matrix(c["a"], 0.01)
            c["dx_t"] = empty(c["x"])
            c["dy_t"] = empty(c["y"]) if c["use_y"] else None
            for n in ("w_pre", "w_post", "gate"):
                c["d" + n] = torch.empty_like(c[n]) if c[n] is not None else None
    elif c["op"] == "clip":
        c["grads"] = [(c["size"] * normal(n)).to(DTYPES[t]) for n, t in _clip_sizes(c)]
        c["flat"], c["out_t"] = _flat_views(c, {t: DTYPES[t] for t in DTYPES}, dev)
        c["norm_t"] = torch.empty(1, device=dev)
    else:
        P, V, T, H = c["P"], c["V"], c["T"], c["H"]
        # the n-th most frequent token comes up about 1 / n of the time; frequent ones lie anywhere in
        # the vocabulary, here with one rank's worth of rows that no rank of the call holds
        n = V * P + (V if c["first"] else 0)
        rank = torch.exp(torch.rand(T, generator=g, device=dev) * math.log(n)).long().clamp_(max=n) - 1
        c["tokens"] = (rank * 2654435761 + 12345) % n
        if c["op"] == "embed":
            c["tables"] = [normal(V, H).to(DTYPES[c["table"]]) for _ in range(P)]
            c["out_t"] = [torch.empty(T, H, dtype=DTYPES[c["out"]], device=dev) for _ in range(P)]
        else:
            c["dout_t"] = (0.01 * normal(T, H)).to(DTYPES[c["out"]])
            c["dtables"] = [torch.empty(V, H, dtype=DTYPES[c["table"]], device=dev) for _ in range(P)]
    return c


# ---- the plain forms -------------------------------------------------------------------------------------


def _rs(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)


def _gate_rows(c):
    """The gate of every row, [T, H] or [1, H]."""
    if c["gate"] is None:
        return 1.0
    gate = c["gate"].float()
    return gate if c["groups"] == 1 else gate.repeat_interleave(c["T"] // c["groups"], 0)


def _norm_plain(c):
    out = c["x_t"]
    if c["use_y"]:
        n = c["y_t"].float()
        if c["post"]:
            n = n * _rs(n) * (c["offset"] + c["w_post"].float())
        out = (c["alpha"] * out.float() + _gate_rows(c) * n).to(out.dtype)
    s = out.float()
    a = (s * _rs(s) * (c["offset"] + c["w_pre"].float())).to(DTYPES[c["a"]])
    return [out if c["use_y"] else None, a]


def _norm_backward_plain(c):
    s, da = c["x_t"].float(), c["da_t"].float()
    rs = _rs(s)
    u = da * (c["offset"] + c["w_pre"].float())
    t = c["dout_t"].float() + rs * u - s * rs ** 3 * (u * s).mean(dim=1, keepdim=True)
    dw_pre = (da * s * rs).sum(0)
    dy = dw_post = dgate = None
    if c["use_y"]:
        y = c["y_t"].float()
        dn = _gate_rows(c) * t
        n, dy = y, dn
        if c["post"]:
            w, ry = c["offset"] + c["w_post"].float(), _rs(y)
            n = y * ry * w
            dw_post = (dn * y * ry).sum(0)
            dy = ry * dn * w - y * ry ** 3 * (dn * w * y).mean(dim=1, keepdim=True)
        if c["gate"] is not None:
            dgate = (t * n).view(c["groups"], -1, c["H"]).sum(1)
    p = DTYPES[c["param"]]
    return [(c["alpha"] * t).to(DTYPES[c["x"]]), None if dy is None else dy.to(DTYPES[c["y"]]), dw_pre.to(p),
            None if dw_post is None else dw_post.to(p), None if dgate is None else dgate.to(p)]


def _clip_plain(c):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in c["grads"]]).sum()
    norm = total.sqrt()
    factor = (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    for t, out in zip(c["grads"], c["out_t"]):
        out.copy_(t.float() * factor)
    return [norm.float().view(1), c["flat"]]


def _embed_plain(c):
    out = []
    for r, table in enumerate(c["tables"]):
        at = c["tokens"] - (c["first"] + r * c["V"])
        here = (at >= 0) & (at < c["V"])
        rows = c["scale"] * table[at.clamp(0, c["V"] - 1)].float()
        out.append(torch.where(here[:, None], rows, 0.0).to(DTYPES[c["out"]]))
    return out


def _embed_backward_plain(c):
    n = c["P"] * c["V"]
    at = c["tokens"] - c["first"]
    here = (at >= 0) & (at < n)
    d = torch.zeros(n, c["H"], device=at.device).index_add_(0, at[here], c["dout_t"][here].float())
    return list((c["scale"] * d).to(DTYPES[c["table"]]).view(c["P"], c["V"], c["H"]))


def run(state):
    c = state
    if own:
        import error_compensated_bit_echo_amd as E

        if c["op"].startswith("norm"):
            same = dict(y=c["y_t"], gate=c["gate"], w_post=c["w_post"], w_pre=c["w_pre"], post_norm=c["post"],
                        residual_scale=c["alpha"], weight_offset=c["offset"], eps=EPS)
            if c["op"] == "norm":
                E.echo_block_norm(c["x_t"], out=c["out_t"], a=c["a_t"], **same)
                return [c["out_t"], c["a_t"]]
            E.echo_block_norm_backward(c["x_t"], dout=c["dout_t"], da=c["da_t"], dx=c["dx_t"], dy=c["dy_t"],
                                       dgate=c["dgate"], dw_post=c["dw_post"], dw_pre=c["dw_pre"], **same)
            return [c["dx_t"], c["dy_t"], c["dw_pre"], c["dw_post"], c["dgate"]]
        if c["op"] == "clip":
            E.echo_clip_grads(c["grads"], c["max_norm"], c["norm_t"], out=c["out_t"])
            return [c["norm_t"], c["flat"]]
        if c["op"] == "embed":
            return E.echo_embed(c["tables"], c["tokens"], c["out_t"], scale=c["scale"], first=c["first"])
        return E.echo_embed_backward(c["dout_t"], c["tokens"], c["dtables"], scale=c["scale"], first=c["first"])
    return {"norm": _norm_plain, "norm backward": _norm_backward_plain, "clip": _clip_plain, "embed": _embed_plain,
            "embed backward": _embed_backward_plain}[c["op"]](c)


# ---- what a pass cannot do without -----------------------------------------------------------------------


def work(case):
    c = case
    size = {k: v.itemsize for k, v in DTYPES.items()}
    if c["op"].startswith("norm"):
        n = c["T"] * c["H"]
        params = c["H"] * size[c["param"]] * (1 + c["post"] + c["groups"])
        x, y, a = size[c["x"]], size[c["y"]] * c["use_y"], size[c["a"]]
        if c["op"] == "norm":
            return {"bytes": n * (x * (1 + c["use_y"]) + y + a) + params, "flops": n * (4 + 6 * c["use_y"])}
        return {"bytes": n * (3 * x + 2 * y + a) + 2 * params, "flops": n * (10 + 12 * c["use_y"])}
    if c["op"] == "clip":
        sizes = _clip_sizes(c)
        return {"bytes": sum(2 * n * size[t] for n, t in sizes) + 4, "flops": 3 * sum(n for n, _ in sizes)}
    P, V, T, H = c["P"], c["V"], c["T"], c["H"]
    if c["op"] == "embed":
        return {"bytes": 8 * T + min(T, P * V) * H * size[c["table"]] + P * T * H * size[c["out"]], "flops": T * H}
    return {"bytes": 8 * T + T * H * size[c["out"]] + P * V * H * size[c["table"]], "flops": 2 * T * H}


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def _exact_rmsnorm(v, w, offset):
    root = torch.sqrt(torch.linalg.vector_norm(v, dim=1, keepdim=True) ** 2 / v.shape[1] + EPS)
    v = v / root
    return v if w is None else v * (w + offset)


def _exact_branch(c, y, gate, w_post):
    n = _exact_rmsnorm(y, w_post, c["offset"]) if c["post"] else y
    if gate is None:
        return n
    return (n.view(c["groups"], -1, c["H"]) * gate[:, None, :]).view(c["T"], c["H"])


def _exact_norm(c):
    wide = {n: None if c[n] is None else c[n].double() for n in ("x_t", "y_t", "gate", "w_post", "w_pre")}
    if not c["use_y"]:
        return [None, _exact_rmsnorm(wide["x_t"], wide["w_pre"], c["offset"])]
    out = c["alpha"] * wide["x_t"] + _exact_branch(c, wide["y_t"], wide["gate"], wide["w_post"])
    stored = out.to(c["x_t"].dtype).double()  # the next block starts from the stream as it is stored
    return [out, _exact_rmsnorm(stored, wide["w_pre"], c["offset"])]


def _exact_norm_backward(c):
    """By differentiating the definition."""
    leaf = {n: None if c[n] is None else c[n].double().requires_grad_() for n in ("x_t", "y_t", "gate", "w_post", "w_pre")}
    a = _exact_rmsnorm(leaf["x_t"], leaf["w_pre"], c["offset"])
    d_stream, dw_pre = torch.autograd.grad(a, [leaf["x_t"], leaf["w_pre"]], c["da_t"].double())
    del a
    d_stream += c["dout_t"].double()
    got = dict.fromkeys(("y_t", "gate", "w_post"))
    if c["use_y"]:
        wrt = [n for n in got if leaf[n] is not None]
        branch = _exact_branch(c, leaf["y_t"], leaf["gate"], leaf["w_post"])
        got.update(zip(wrt, torch.autograd.grad(branch, [leaf[n] for n in wrt], d_stream)))
    return [c["alpha"] * d_stream, got["y_t"], dw_pre, got["w_post"], got["gate"]]


def _exact_clip(c):
    norm = math.sqrt(math.fsum(torch.linalg.vector_norm(t.double()).item() ** 2 for t in c["grads"]))
    factor = min(1.0, c["max_norm"] / (norm + 1e-6))
    flat, out = _flat_views(c, dict.fromkeys(DTYPES, torch.float64), c["norm_t"].device)
    for o, t in zip(out, c["grads"]):
        torch.mul(t.double(), factor, out=o)
    return [torch.tensor([norm], dtype=torch.float64, device=c["norm_t"].device), flat]


def _exact_embed(c):
    V, P, H = c["V"], c["P"], c["H"]
    out = [torch.zeros(c["T"], H, dtype=torch.float64, device=c["tokens"].device) for _ in range(P)]
    owner = torch.div(c["tokens"] - c["first"], V, rounding_mode="floor")
    for r in range(P):
        t = (owner == r).nonzero().view(-1)
        out[r][t] = c["tables"][r][c["tokens"][t] - c["first"] - r * V].double() * c["scale"]
    return out


def _exact_embed_backward(c):
    """Runs of equal tokens in sorted order, as differences of running sums of few rows at a time."""
    V, P, H = c["V"], c["P"], c["H"]
    d = torch.zeros(P * V, H, dtype=torch.float64, device=c["tokens"].device)
    at, order = torch.sort(c["tokens"] - c["first"], stable=True)
    ids, counts = torch.unique_consecutive(at, return_counts=True)
    ends = counts.cumsum(0)
    for lo in range(0, H, 512):  # a few columns at a time
        sums = c["dout_t"][:, lo:lo + 512][order].double().cumsum(0)
        rows = sums[ends - 1]
        rows[1:] -= sums[ends[:-1] - 1]
        held = (ids >= 0) & (ids < P * V)
        d[ids[held], lo:lo + 512] = rows[held] * c["scale"]
    return list(d.view(P, V, H))


def exact(case, seed):
    c = prepare(case, seed)
    return {"norm": _exact_norm, "norm backward": _exact_norm_backward, "clip": _exact_clip, "embed": _exact_embed,
            "embed backward": _exact_embed_backward}[c["op"]](c)
