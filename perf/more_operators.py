"""What joins gated blocks into a network and their gradients to the optimizer,
measured: the norms behind and in front of a block fused with its gate and the
residual sum (forward and backward), the global norm of many gradients, and
their clipping.

Each case is computed in plain torch operations, or, where `own` is set, by
the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = dict(bf16=torch.bfloat16, fp32=torch.float32)
EPS = 1e-5
DECAY = 0.97  # of the clipping bound from pass to pass


def listed():
    return [
        # between two blocks of a decode step: eight tokens, latency counts
        dict(name="join decode 8 rows", op="join", R=8, C=2048, x="bf16", b="bf16", y="bf16", post="rms",
             kind="rms", bias=False, gate=0, xs=1.0, bs=1.0),
        # the training step's join of two 2048-wide blocks, a learned gate per channel
        dict(name="join train 8192x2048", op="join", R=8192, C=2048, x="bf16", b="bf16", y="bf16", post="rms",
             kind="rms", bias=False, gate=8192, xs=1.0, bs=1.0),
        # the 5120-wide block with its residual stream in fp32, layer norms on both sides
        dict(name="join wide fp32 stream", op="join", R=16384, C=5120, x="fp32", b="bf16", y="bf16",
             post="layer", kind="layer", bias=True, gate=16384, xs=1.0, bs=0.5),
        # a ragged batch of odd width, one row of gates per sequence, no norm behind the block
        dict(name="join odd sequences", op="join", R=1999, C=1111, x="fp32", b="fp32", y="fp32", post="none",
             kind="layer", bias=True, gate=257, xs=1.0, bs=1.0),
        # the gradients of the training step's join
        dict(name="join grad 8192x2048", op="join_grad", R=8192, C=2048, x="bf16", b="bf16", y="bf16",
             post="rms", kind="rms", bias=False, gate=8192, xs=1.0, bs=1.0),
        # of the wide block's with the fp32 stream
        dict(name="join grad wide fp32 stream", op="join_grad", R=16384, C=5120, x="fp32", b="bf16", y="bf16",
             post="layer", kind="layer", bias=True, gate=16384, xs=1.0, bs=0.5),
        # of the ragged batch, gates' gradients summed per sequence
        dict(name="join grad odd sequences", op="join_grad", R=1999, C=1111, x="fp32", b="fp32", y="fp32",
             post="layer", kind="layer", bias=True, gate=257, xs=1.0, bs=1.0),
        # adapters, norms, biases: many small gradients behind each other in one buffer
        dict(name="norm 150 small tensors", op="norm", grad="fp32", tensors=150, most=9000, order="two"),
        # the gradients of five 2048-wide blocks in fp32
        dict(name="norm 173M fp32", op="norm", grad="fp32", tensors=20, most=11534336, order="two"),
        # the wide block's, matrices in bf16 and vectors in fp32, the largest magnitude
        dict(name="norm 212M mixed largest", op="norm", grad="mixed", tensors=4, most=70778880, order="max"),
        # clipping the small ones in place
        dict(name="clip 40 small tensors", op="clip", grad="fp32", tensors=40, most=5000, order="two"),
        # and the wide block's
        dict(name="clip 212M mixed", op="clip", grad="mixed", tensors=4, most=70778880, order="two"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("join", "join_grad", "norm", "clip"))
    if op in ("join", "join_grad"):
        C = log(8, 13824)
        R = log(1, min(16384, 16384 * 5120 // C))
        gate = rng.choice((0, 1, R, log(1, R)))  # rows that share a row of gates; 0: none
        return dict(op=op, R=R, C=C, x=rng.choice(("bf16", "fp32")), b=rng.choice(("bf16", "fp32")),
                    y=rng.choice(("bf16", "fp32")), post=rng.choice(("none", "layer", "rms")),
                    kind=rng.choice(("layer", "rms")), bias=rng.random() < 0.5, gate=gate,
                    xs=rng.choice((1.0, 0.75)), bs=rng.choice((1.0, 0.22)))
    tensors = log(1, 300)
    return dict(op=op, grad=rng.choice(("bf16", "fp32", "mixed")), tensors=tensors,
                most=log(100, 170e6 / tensors), order=rng.choice(("two", "max")))


# ---- what a program has in hand ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, sd=1.0):
    return torch.randn(shape, generator=g, device=DEV) * sd


def _rows(g, R, C):
    """Hidden-state rows: an offset, and a few channels much larger than the rest."""
    ch = torch.ones(C, device=DEV)
    ch[torch.rand(C, generator=g, device=DEV) < 0.01] = 8.0
    return _normal(g, R, C) * ch + _normal(g, C, sd=0.1)


def _sizes(case):
    """Elements of each tensor: matrices, then vectors."""
    n, most = case["tensors"], case["most"]
    many = max(1, (3 * n) // 4)
    sizes = [max(1, most - (i % 5) * (most // 7)) if n > 25 else most for i in range(many)]
    return sizes, [min(most, 2048 + 37 * i) for i in range(n - many)]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("norm", "clip"):
        # tensors of one type lie behind each other in one buffer, as a reduction over ranks leaves them
        mats, vecs = _sizes(case)
        parts = [mats, vecs] if case["grad"] == "mixed" else [mats + vecs]
        types = [torch.bfloat16, torch.float32] if case["grad"] == "mixed" else [TYPES[case["grad"]]]
        parts = [p for p in parts if p]
        s["flat"] = [_normal(g, sum(p), sd=1e-3).to(t) for p, t in zip(parts, types)]
        s["bound"] = 5e-4 * math.sqrt(sum(mats) + sum(vecs)) if case["order"] == "two" else 1e-3
        if own:
            import mxfp4_block_scaled_fp4q_amd as fq
            s["plan"] = fq.grad_plan([t for f, p in zip(s["flat"], parts) for t in f.split(p)])
        return s
    R, C = case["R"], case["C"]
    s["x"], s["b"] = _rows(g, R, C).to(TYPES[case["x"]]), _rows(g, R, C).to(TYPES[case["b"]])
    s["w"] = 1.0 + _normal(g, C, sd=0.1)
    s["c"] = _normal(g, C, sd=0.1) if case["bias"] else None
    post = case["post"] != "none"
    s["pw"] = 0.5 + _normal(g, C, sd=0.1) if post else None
    s["pc"] = _normal(g, C, sd=0.1) if post and case["bias"] else None
    s["gate"] = None
    if case["gate"]:
        s["gate"] = _normal(g, -(-R // case["gate"]), C, sd=0.5).to(TYPES[case["b"]])
    if case["op"] == "join_grad":
        s["dy"] = _normal(g, R, C, sd=1e-3).to(TYPES[case["y"]])
        s["dxo"] = _normal(g, R, C, sd=1e-3).to(TYPES[case["x"]])
        s["xo"], _, s["stats"] = _forward(s)
        del s["x"]
    return s


# ---- the plain forms ----

def _standard(x, kind):
    """x normalised along its rows, with the mean and the reciprocal deviation."""
    mean = x.mean(1) if kind == "layer" else None
    d = x if mean is None else x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + EPS)
    return d * rstd[:, None], mean, rstd


def _gates(s, rows):
    """The gate of every row, or one row for all."""
    gate = s["gate"].float()
    if gate.shape[0] == 1:
        return gate
    return gate[torch.arange(rows, device=DEV) // s["case"]["gate"]]


def _group_sums(t, rows):
    """Sums over each `rows` rows; the last group may be shorter."""
    short = -t.shape[0] % rows
    if short:
        t = torch.cat((t, t.new_zeros(short, t.shape[1])))
    return t.view(-1, rows, t.shape[1]).sum(1)


def _forward(s):
    c = s["case"]
    n, stats = s["b"].float(), (None, None)
    if c["post"] != "none":
        n, *stats = _standard(n, c["post"])
        n = n * s["pw"]
        if s["pc"] is not None:
            n = n + s["pc"]
    if s["gate"] is not None:
        n = n * _gates(s, c["R"])
    x = c["xs"] * s["x"].float() + c["bs"] * n
    y, mean, rstd = _standard(x, c["kind"])
    y = y * s["w"]
    if s["c"] is not None:
        y = y + s["c"]
    return x.to(s["x"].dtype), y.to(TYPES[c["y"]]), (*stats, mean, rstd)


def _join(s):
    x, y, (pm, pr, mean, rstd) = _forward(s)
    return dict(x=x, y=y, post_mean=pm, post_rstd=pr, mean=mean, rstd=rstd)


def _back(t, xh, rstd, layer):
    d = t - xh * (t * xh).mean(1, keepdim=True)
    if layer:
        d = d - t.mean(1, keepdim=True)
    return d * rstd[:, None]


def _join_grad(s):
    c = s["case"]
    pm, pr, mean, rstd = s["stats"]
    x, dy = s["xo"].float(), s["dy"].float()
    xh = (x if mean is None else x - mean[:, None]) * rstd[:, None]
    out = dict(d_weight=(dy * xh).sum(0), d_bias=dy.sum(0) if c["bias"] else None)
    d = s["dxo"].float() + _back(dy * s["w"], xh, rstd, c["kind"] == "layer")
    out["dx"] = (c["xs"] * d).to(s["dxo"].dtype)
    post, n = c["post"] != "none", s["b"].float()
    if post:
        h = n = (n if pm is None else n - pm[:, None]) * pr[:, None]
        n = n * s["pw"]
        if s["pc"] is not None:
            n = n + s["pc"]
    e = c["bs"] * d
    if s["gate"] is not None:
        out["d_gate"] = _group_sums(e * n, c["gate"])
        e = e * _gates(s, c["R"])
    if post:
        out["d_post_weight"] = (e * h).sum(0)
        out["d_post_bias"] = e.sum(0) if s["pc"] is not None else None
        e = _back(e * s["pw"], h, pr, c["post"] == "layer")
    out["db"] = e.to(s["b"].dtype)
    return out


def _norm_of(s):
    if s["case"]["order"] == "max":
        return torch.stack([f.abs().max().float() for f in s["flat"]]).max()
    return torch.stack([f.float().square().sum() for f in s["flat"]]).sum().sqrt()


def _scale_of(norm, bound):
    return (bound / (norm + 1e-6)).clamp(max=1.0)


def _norm(s):
    norm = _norm_of(s)
    return dict(norm=norm, scale=_scale_of(norm, s["bound"]))


def _next_bound(s):
    """The bound falls from pass to pass, so that gradients that a pass has
    clipped are clipped by the next one too."""
    s["bound"] *= DECAY
    return s["bound"]


def _clip(s):
    norm = _norm_of(s)
    scale = _scale_of(norm, _next_bound(s))
    for f in s["flat"]:
        f.copy_(f.float() * scale)
    return dict(norm=norm, grads=s["flat"])


# ---- the library's calls ----

def _library(s):
    import mxfp4_block_scaled_fp4q_amd as fq
    c = s["case"]
    kinds = dict(none=fq.NO_NORM, layer=fq.LAYER_NORM, rms=fq.RMS_NORM)
    if c["op"] in ("norm", "clip"):
        order = fq.NORM_MAX if c["order"] == "max" else fq.NORM_L2
        if c["op"] == "norm":
            norm, scale = fq.grad_norm(s["plan"], s["bound"], order=order)
            return dict(norm=norm, scale=scale)
        return dict(norm=fq.clip_grads(s["plan"], _next_bound(s), order=order), grads=s["flat"])
    how = dict(kind=kinds[c["kind"]], post_kind=kinds[c["post"]], post_weight=s["pw"], post_bias=s["pc"],
               gate=s["gate"], gate_rows=c["gate"] or None, x_scale=c["xs"], branch_scale=c["bs"])
    if c["op"] == "join":
        x, y, (pm, pr, mean, rstd) = fq.residual_norm(s["x"], s["b"], s["w"], s["c"], eps=EPS,
                                                      out_dtype=TYPES[c["y"]], **how)
        return dict(x=x, y=y, post_mean=pm, post_rstd=pr, mean=mean, rstd=rstd)
    r = fq.residual_norm_grad(s["dy"], s["dxo"], s["xo"], s["b"], s["stats"], s["w"], want_bias=c["bias"], **how)
    return dict(zip(("dx", "db", "d_weight", "d_bias", "d_post_weight", "d_post_bias", "d_gate"), r))


def run(state):
    if own:
        return _library(state)
    return dict(join=_join, join_grad=_join_grad, norm=_norm, clip=_clip)[state["case"]["op"]](state)


def work(case):
    if case["op"] in ("norm", "clip"):
        mats, vecs = _sizes(case)
        size = 2 if case["grad"] == "bf16" else 4
        moved = sum(mats) * (4 if case["grad"] == "fp32" else 2) + sum(vecs) * size
        n = sum(mats) + sum(vecs)
        return dict(bytes=moved * (2 if case["op"] == "clip" else 1), flops=n * (3.0 if case["op"] == "clip" else 2.0))
    R, C = case["R"], case["C"]
    x, b, y = (2 if case[k] == "bf16" else 4 for k in "xby")
    post, gate = case["post"] != "none", -(-R // case["gate"]) if case["gate"] else 0
    vectors = (1 + post) * (2 if case["bias"] else 1)
    means = (case["kind"] == "layer") + (case["post"] == "layer")
    stats = 4 * R * (1 + post + means)
    if case["op"] == "join":
        return dict(bytes=R * C * (2 * x + b + y) + gate * C * b + 4 * C * vectors + stats,
                    flops=R * C * (12.0 + 8.0 * post))
    # the biases are not read, all vectors but those of ones get a gradient
    return dict(bytes=R * C * (3 * x + 2 * b + y) + gate * C * (b + 4) + 4 * C * (vectors + 1 + post) + stats,
                flops=R * C * (18.0 + 18.0 * post))


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    s.pop("plan", None)
    d = torch.float64
    if case["op"] in ("norm", "clip"):
        flat = [f.to(d) for f in s["flat"]]
        if case["order"] == "max":
            norm = max(float(f.max().maximum(-f.min())) for f in flat)
        else:
            norm = math.sqrt(sum(float(torch.dot(f, f)) for f in flat))
        bound = s["bound"] * (DECAY if case["op"] == "clip" else 1.0)
        scale = min(1.0, bound / (norm + 1e-6))
        whole = torch.tensor(norm, dtype=d, device=DEV)
        if case["op"] == "norm":
            return dict(norm=whole, scale=torch.tensor(scale, dtype=d, device=DEV))
        return dict(norm=whole, grads=[f * scale for f in flat])

    R, C = case["R"], case["C"]
    w, cb, pw, pc, b, gate = (None if s[k] is None else s[k].to(d) for k in ("w", "c", "pw", "pc", "b", "gate"))
    group = torch.arange(R, device=DEV).div(case["gate"] or R, rounding_mode="floor")
    rows = torch.ones(1, C, dtype=d, device=DEV) if gate is None else gate

    def centre(t, kind):
        return t - t.sum(1, keepdim=True) / C if kind == "layer" else t

    def spread(t):
        return (torch.linalg.vector_norm(t, dim=1) ** 2 / C + EPS) ** -0.5

    if case["op"] == "join":
        n, pm, pr = b, None, None
        if case["post"] != "none":
            t = centre(b, case["post"])
            pm, pr = (b.sum(1) / C if case["post"] == "layer" else None), spread(t)
            n = torch.einsum("rc,r,c->rc", t, pr, pw)
            n = n if pc is None else n + pc
        x = case["xs"] * s["x"].to(d) + case["bs"] * rows[group] * n
        t = centre(x, case["kind"])
        r = spread(t)
        y = torch.einsum("rc,r,c->rc", t, r, w)
        return dict(x=x, y=y if cb is None else y + cb, post_mean=pm, post_rstd=pr,
                    mean=x.sum(1) / C if case["kind"] == "layer" else None, rstd=r)

    pm, pr, m, r = (None if t is None else t.to(d)[:, None] for t in s["stats"])
    x, dy = s["xo"].to(d), s["dy"].to(d)
    xh = (x - (0.0 if m is None else m)) * r
    t = dy * w
    rest = t.sum(1, keepdim=True) / C if case["kind"] == "layer" else 0.0
    whole = s["dxo"].to(d) + r * (t - rest - xh * ((t * xh).sum(1, keepdim=True) / C))
    out = dict(dx=case["xs"] * whole, d_weight=(dy * xh).sum(0), d_bias=dy.sum(0) if case["bias"] else None)
    e = case["bs"] * whole
    h = b if pr is None else (b - (0.0 if pm is None else pm)) * pr
    if gate is not None:
        n = h if pw is None else h * pw if pc is None else h * pw + pc
        out["d_gate"] = torch.stack([p.sum(0) for p in (e * n).split(case["gate"])])
    e = e * rows[group]
    if pr is None:
        return dict(out, db=e)
    out["d_post_weight"], out["d_post_bias"] = (e * h).sum(0), e.sum(0) if pc is not None else None
    u = e * pw
    rest = u.sum(1, keepdim=True) / C if case["post"] == "layer" else 0.0
    return dict(out, db=pr * (u - rest - h * ((u * h).sum(1, keepdim=True) / C)))
