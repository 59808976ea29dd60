"""The operators of one training step of a gated feed-forward block in MXFP4,
measured: the gated projections (forward, and the gradient that leaves the
activation), the norm in front of them (forward and backward) and the AdamW
step over the block's tensors.

Each case is computed in plain torch operations, or, where `own` is set, by
the library's calls.  Operands of the products are held as E2M1 codes with one
E8M0 scale byte per 32 elements, as the quantiser writes them; the 8-bit
optimizer states are E4M3 values with one E8M0 scale per 32.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GELU_A, GELU_B = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # one token of one request through a 2048-wide block: weights from memory, latency counts
        dict(name="gated decode 1 token", op="gated", M=1, F=5632, K=2048, act="silu", save=False),
        # the training step's forward: 8192 tokens, gate and up kept for the backward pass
        dict(name="gated train 8192 tokens", op="gated", M=8192, F=5632, K=2048, act="silu", save=True),
        # a long prompt batch through a 5120-wide block, nothing kept
        dict(name="gated prompt 16384 wide", op="gated", M=16384, F=13824, K=5120, act="silu", save=False),
        # the training step's backward: the gradient behind the down projection, through the activation
        dict(name="gated grad 8192 tokens", op="gated_grad", M=8192, F=5632, K=2048, act="silu"),
        # a ragged micro-batch of a small block: odd tokens, odd width, a half step at the end of K
        dict(name="gated grad ragged", op="gated_grad", M=1237, F=1407, K=960, act="gelu"),
        # the norm in front of a decode step: eight rows, latency counts
        dict(name="norm decode 8 rows", op="norm", R=8, C=2048, kind="rms", dtype="bf16", bias=False),
        # the training step's norm
        dict(name="norm train 8192x2048", op="norm", R=8192, C=2048, kind="layer", dtype="bf16", bias=True),
        # its backward at the wide block's size
        dict(name="norm grad 16384x5120", op="norm_grad", R=16384, C=5120, kind="layer", dtype="bf16", bias=True),
        # fp32 activations of a ragged batch with an odd width
        dict(name="norm grad odd fp32", op="norm_grad", R=1999, C=1111, kind="rms", dtype="fp32", bias=False),
        # many small tensors (adapters, norms, biases): launches count
        dict(name="adamw 150 small tensors", op="adamw", bits=32, grad="fp32", tensors=150, most=9000, copy=True),
        # the 2048-wide block's tensors of five layers, 32-bit states, the bf16 copy that is quantised next
        dict(name="adamw 32-bit 173M", op="adamw", bits=32, grad="fp32", tensors=20, most=11534336, copy=True),
        # the 5120-wide block's three matrices and its norm, 8-bit states, bf16 gradients
        dict(name="adamw 8-bit 212M", op="adamw", bits=8, grad="bf16", tensors=4, most=70778880, copy=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("gated", "gated_grad", "norm", "norm_grad", "adamw"))
    if op in ("gated", "gated_grad"):
        case = dict(op=op, M=log(1, 16384), F=log(32, 13824), K=64 * log(2, 80),
                    act=rng.choice(("silu", "gelu")))
        return dict(case, save=rng.random() < 0.5) if op == "gated" else case
    if op in ("norm", "norm_grad"):
        return dict(op=op, R=log(1, 16384), C=log(8, 13824), kind=rng.choice(("layer", "rms")),
                    dtype=rng.choice(("bf16", "fp32")), bias=rng.random() < 0.5)
    tensors = log(1, 300)
    return dict(op=op, bits=rng.choice((8, 32)), grad=rng.choice(("bf16", "fp32")), tensors=tensors,
                most=log(100, 180e6 / tensors), copy=rng.random() < 0.5)


# ---- what a program has in hand ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, sd=1.0):
    return torch.randn(shape, generator=g, device=DEV) * sd


def _quantise(x):
    """Codes [R, K/2] and scale bytes [R, K/32] of rows of x, to nearest."""
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    byte = ((b.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp(min=0)
    m = b.abs() / (byte << 23).view(torch.float32)[..., None]
    edges = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=DEV)
    code = torch.bucketize(m, edges).to(torch.uint8) + (b < 0).to(torch.uint8) * 8
    code = code.reshape(R, K // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), byte.to(torch.uint8).contiguous()


def _act_rows(g, R, C):
    """Hidden-state rows: an offset, and a few channels much larger than the rest."""
    ch = torch.ones(C, device=DEV)
    ch[torch.rand(C, generator=g, device=DEV) < 0.01] = 8.0
    return _normal(g, R, C) * ch + _normal(g, C, sd=0.1)


def _sizes(case):
    """Elements of each tensor, the decayed ones (the first `nd`) before the others."""
    n, most = case["tensors"], case["most"]
    many = max(1, (3 * n) // 4)  # matrices; the rest are vectors
    sizes = [max(1, most - (i % 5) * (most // 7)) if n > 25 else most for i in range(many)]
    sizes += [min(most, 2048 + 37 * i) for i in range(n - many)]
    return sizes, many


def _places(sizes):
    """First element of each tensor in the flat buffers (whole blocks of 32), and their length."""
    at, places = 0, []
    for s in sizes:
        places.append(at)
        at += -(-s // 32) * 32
    return places, at


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        if op == "gated":
            s["x"] = _quantise(_act_rows(g, M, K))
            s["w"] = _quantise(_normal(g, 2 * F, K, sd=0.02))  # gate rows, then up rows
        else:
            s["dy"] = _quantise(_normal(g, M, K, sd=1e-3))
            s["wd"] = _quantise(_normal(g, F, K, sd=0.02))
            s["gu"] = _normal(g, M, 2 * F, sd=1.0).bfloat16()
        return s
    if op in ("norm", "norm_grad"):
        R, C = case["R"], case["C"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = _act_rows(g, R, C).to(dt)
        s["x"], s["eps"] = x, 1e-5
        s["weight"] = 1.0 + _normal(g, C, sd=0.1)
        s["bias"] = _normal(g, C, sd=0.1) if case["bias"] else None
        if op == "norm_grad":
            s["dy"] = _normal(g, R, C, sd=1e-3).to(dt)
            xf = x.float()
            s["mean"] = xf.mean(1) if case["kind"] == "layer" else None
            c = xf - s["mean"][:, None] if case["kind"] == "layer" else xf
            s["rstd"] = (c.square().mean(1) + s["eps"]).rsqrt()
        return s
    sizes, many = _sizes(case)
    places, n = _places(sizes)
    real = torch.zeros(n, dtype=torch.bool, device=DEV)
    for a, k in zip(places, sizes):
        real[a:a + k] = True
    s.update(hyper=dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=100, seed=1234), wd=0.1,
             nd=places[many] if many < len(sizes) else n)
    s["p"] = _normal(g, n, sd=0.02) * real
    s["g"] = (_normal(g, n, sd=1e-3) * real).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
    m, r = _normal(g, n, sd=3e-4) * real, (_normal(g, n, sd=1e-3).abs() + 1e-6) * real
    s["copy"] = s["p"].bfloat16() if case["copy"] else None
    if case["bits"] == 32:
        s["m"], s["v"], s["ms"], s["vs"] = m, r.square(), None, None
    else:
        half = torch.full((n,), 0x8000, dtype=torch.int32, device=DEV)
        s["m"], s["ms"] = _to_e4m3(m, half)
        s["v"], s["vs"] = _to_e4m3(r, half)
    if own:
        import mxfp4_block_scaled_fp4q_amd as fq

        def cut(t, block=1):
            return None if t is None else [t[a // block:a // block + -(-k // block)]
                                           for a, k in zip(places, sizes)]
        s["plan"] = fq.adamw_plan(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]), cut(s["ms"], 32),
                                  cut(s["vs"], 32), copies=cut(s["copy"]),
                                  weight_decay=[s["wd"] if i < many else 0.0 for i in range(len(sizes))])
    return s


# ---- the plain forms ----

def _values(q):
    """fp32 values of (codes, scale bytes)."""
    codes, byte = q
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).reshape(codes.shape[0], -1, 32)
    return (v * (byte.int() << 23).view(torch.float32)[..., None]).flatten(1)


def _sigmoid_of(x, act):
    z = x if act == "silu" else GELU_A * (x + GELU_B * x * x * x)
    return 1.0 / (1.0 + torch.exp(-z))


def _slope_of(x, act):
    return 1.0 if act == "silu" else GELU_A * (1.0 + 3.0 * GELU_B * x * x)


def _gated(s):
    c = s["case"]
    y = _values(s["x"]) @ _values(s["w"]).T
    g, u = y[:, :c["F"]], y[:, c["F"]:]
    h = (g * _sigmoid_of(g, c["act"]) * u).bfloat16()
    return dict(h=h, gate=g.bfloat16(), up=u.bfloat16()) if c["save"] else dict(h=h)


def _gated_grad(s):
    c = s["case"]
    dh = _values(s["dy"]) @ _values(s["wd"]).T
    g, u = s["gu"][:, :c["F"]].float(), s["gu"][:, c["F"]:].float()
    sg = _sigmoid_of(g, c["act"])
    d = sg + g * sg * (1.0 - sg) * _slope_of(g, c["act"])
    return dict(d_gate=(dh * u * d).bfloat16(), d_up=(dh * g * sg).bfloat16())


def _norm(s):
    x = s["x"].float()
    mean = x.mean(1) if s["case"]["kind"] == "layer" else None
    if mean is not None:
        x = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(x.square().mean(1) + s["eps"])
    y = x * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    layer = s["case"]["kind"] == "layer"
    xh = (x - s["mean"][:, None] if layer else x) * s["rstd"][:, None]
    t = dy * s["weight"]
    dx = t - xh * (t * xh).mean(1, keepdim=True)
    if layer:
        dx = dx - t.mean(1, keepdim=True)
    dx = (dx * s["rstd"][:, None]).to(s["x"].dtype)
    return dict(dx=dx, d_weight=(dy * xh).sum(0), d_bias=dy.sum(0) if s["bias"] is not None else None)


def _philox(n, step, seed):
    """32 random bits for each of n positions: Philox4x32-10, counter
    (position / 4, step, 0), word position % 4, key the seed."""
    low = 0xFFFFFFFF
    at = torch.arange(-(-n // 4), device=DEV)
    c0, c1, c2, c3 = at & low, at >> 32, torch.full_like(at, step), torch.zeros_like(at)
    k0, k1 = seed & low, seed >> 32

    def halves(c, m):  # both halves of a 32 x 32 bit product, in 16-bit pieces
        a, b = c & 0xFFFF, c >> 16
        t = a * m
        u = b * m + (t >> 16)
        return u >> 16, ((u & 0xFFFF) << 16) | (t & 0xFFFF)

    def once(c0, c1, c2, c3, k0, k1):
        h0, l0 = halves(c0, 0xD2511F53)
        h1, l1 = halves(c2, 0xCD9E8D57)
        return h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0

    for r in range(10):
        c0, c1, c2, c3 = once(c0, c1, c2, c3, (k0 + r * 0x9E3779B9) & low, (k1 + r * 0xBB67AE85) & low)
    return torch.stack((c0, c1, c2, c3), 1).flatten()[:n]


def _to_e4m3(x, u):
    """x in blocks of 32 as E4M3 codes and E8M0 bytes (largest magnitude in
    [128, 256)), rounded up where the 16 bits u carry past the dropped fraction."""
    b = x.reshape(-1, 32)
    byte = ((b.abs().amax(1).view(torch.int32) >> 23) - 7).clamp(min=0)
    y = b.abs() * ((254 - byte) << 23).view(torch.float32)[:, None]
    u = u.reshape(-1, 32).int()
    normal = ((y.view(torch.int32) + (u << 4)) & ~0xFFFFF).view(torch.float32)
    q = y * 512.0
    low = torch.floor(q)
    low = (low + (torch.floor((q - low) * 65536.0).int() + u >= 65536)) / 512.0
    y = torch.copysign(torch.where(y >= 2.0 ** -6, normal, low), b)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(), byte.to(torch.uint8)


def _from_e4m3(codes, byte):
    # the scales here are far from the ends of the exponent range
    scale = (byte.int() << 23).view(torch.float32)
    return (codes.view(torch.float8_e4m3fn).float().reshape(-1, 32) * scale[:, None]).flatten()


def _adamw(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    g = s["g"].float()
    m = _from_e4m3(s["m"], s["ms"]) if eight else s["m"]
    v = _from_e4m3(s["v"], s["vs"]).square() if eight else s["v"]
    m = h["beta1"] * m + (1.0 - h["beta1"]) * g
    v = h["beta2"] * v + (1.0 - h["beta2"]) * g * g
    root = torch.sqrt(v)
    up = (m / (1.0 - h["beta1"] ** h["step"])) / (root / math.sqrt(1.0 - h["beta2"] ** h["step"]) + h["eps"])
    s["p"][:s["nd"]] *= 1.0 - h["lr"] * s["wd"]
    s["p"] -= h["lr"] * up
    if s["copy"] is not None:
        s["copy"].copy_(s["p"])
    if eight:
        bits = _philox(m.numel(), h["step"], h["seed"])
        for name, x, u in (("m", m, bits & 0xFFFF), ("v", root, bits >> 16)):
            codes, byte = _to_e4m3(x, u)
            s[name].copy_(codes)
            s[name + "s"].copy_(byte)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    out = dict(p=s["p"], copy=s["copy"])
    if s["case"]["bits"] == 8:  # the values that codes and scale bytes stand for
        return dict(out, m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn),
                    m_scale=s["ms"].view(torch.float8_e8m0fnu), v_scale=s["vs"].view(torch.float8_e8m0fnu))
    return dict(out, m=s["m"], v=s["v"])


# ---- the library's calls ----

def _library(s):
    import mxfp4_block_scaled_fp4q_amd as fq
    c = s["case"]
    if c["op"] == "gated":
        (xc, xs), (wc, ws), F = s["x"], s["w"], c["F"]
        r = fq.gemm_gated(xc, xs, wc[:F], ws[:F], wc[F:], ws[F:], act=_act(fq, c), save=c["save"])
        return dict(zip(("h", "gate", "up"), r)) if c["save"] else dict(h=r)
    if c["op"] == "gated_grad":
        F = c["F"]
        r = fq.gemm_gated_grad(*s["dy"], *s["wd"], s["gu"][:, :F], s["gu"][:, F:], act=_act(fq, c))
        return dict(zip(("d_gate", "d_up"), r))
    kind = fq.LAYER_NORM if c.get("kind") == "layer" else fq.RMS_NORM
    if c["op"] == "norm":
        y, mean, rstd = fq.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], kind=kind)
        return dict(y=y, mean=mean, rstd=rstd)
    if c["op"] == "norm_grad":
        r = fq.layer_norm_grad(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=kind,
                               want_bias=s["bias"] is not None)
        return dict(zip(("dx", "d_weight", "d_bias"), r))
    fq.adamw_step(s["plan"], **s["hyper"])
    return _adamw_out(s)


def _act(fq, c):
    return fq.SILU if c["act"] == "silu" else fq.GELU


def run(state):
    if own:
        return _library(state)
    plain = dict(gated=_gated, gated_grad=_gated_grad, norm=_norm, norm_grad=_norm_grad, adamw=_adamw)
    return plain[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("gated", "gated_grad"):
        M, F, K = case["M"], case["F"], case["K"]
        n = 2 * F if op == "gated" else F
        operands = (M + n) * (K / 2 + K / 32)
        if op == "gated":
            moved = M * F * 2 * (3 if case["save"] else 1)
        else:
            moved = M * F * 2 * 4  # gate and up in, their gradients out
        return dict(bytes=operands + moved, flops=2.0 * M * n * K + 10.0 * M * F)
    if op in ("norm", "norm_grad"):
        R, C, e = case["R"], case["C"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            return dict(bytes=R * C * 2 * e + 4 * C * (2 if case["bias"] else 1) +
                        4 * R * (2 if case["kind"] == "layer" else 1), flops=8.0 * R * C)
        return dict(bytes=R * C * 3 * e + 4 * C * (3 if case["bias"] else 2) +
                    4 * R * (2 if case["kind"] == "layer" else 1), flops=14.0 * R * C)
    n = sum(_sizes(case)[0])
    each = 8 + (2 if case["grad"] == "bf16" else 4) + (2 if case["copy"] else 0)
    each += 16 if case["bits"] == 32 else 4 + 4 / 32
    return dict(bytes=n * each, flops=n * (16.0 if case["bits"] == 32 else 60.0))


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    s.pop("plan", None)
    d, op = torch.float64, case["op"]

    def pow2(e):  # of whole numbers, from the bits of the format
        return ((e.long() + 1023) << 52).view(d)

    def read(q):  # sign, two exponent bits, one mantissa bit
        codes, byte = q
        c = torch.stack((codes % 16, codes // 16), 2).flatten(1)
        e, m = ((c // 2) % 4).to(d), (c % 2).to(d)
        v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * pow2(e - 1))
        return torch.where(c >= 8, -v, v) * pow2(byte.long() - 127).repeat_interleave(32, 1)

    def act(x):
        if case["act"] == "silu":
            return x * torch.special.expit(x)
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))

    def act_slope(x):
        if case["act"] == "silu":
            e = torch.special.expit(x)
            return e * (1 + x * (1 - e))
        t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x ** 2)

    if op == "gated":
        x, w, F = read(s["x"]), read(s["w"]), case["F"]
        g, u = x @ w[:F].T, x @ w[F:].T
        h = act(g) * u
        return dict(h=h, gate=g, up=u) if case["save"] else dict(h=h)
    if op == "gated_grad":
        dh, (g, u) = read(s["dy"]) @ read(s["wd"]).T, s["gu"].to(d).split(case["F"], 1)
        return dict(d_gate=dh * u * act_slope(g), d_up=dh * act(g))
    if op == "norm":
        x = s["x"].to(d)
        mean = x.sum(1) / case["C"] if case["kind"] == "layer" else None
        x = x if mean is None else x - mean[:, None]
        rstd = ((x * x).sum(1) / case["C"] + s["eps"]) ** -0.5
        y = torch.einsum("rc,r,c->rc", x, rstd, s["weight"].to(d))
        return dict(y=y if s["bias"] is None else y + s["bias"].to(d), mean=mean, rstd=rstd)
    if op == "norm_grad":
        x, dy, w, r = (s[k].to(d) for k in ("x", "dy", "weight", "rstd"))
        layer = case["kind"] == "layer"
        xh = (x - s["mean"].to(d)[:, None]) * r[:, None] if layer else x * r[:, None]
        t = dy * w
        inner = (t * xh).sum(1, keepdim=True) / case["C"]
        shift = t.sum(1, keepdim=True) / case["C"] if layer else 0.0
        return dict(dx=r[:, None] * (t - shift - xh * inner), d_weight=(dy * xh).sum(0),
                    d_bias=dy.sum(0) if s["bias"] is not None else None)

    h, eight = s["hyper"], case["bits"] == 8

    def state(name):
        if not eight:
            return s[name].to(d)
        return s[name].view(torch.float8_e4m3fn).to(d) * pow2(s[name + "s"].long() - 127).repeat_interleave(32)

    def stored(x, u):  # E4M3 value and scale of each block, rounded by the 16 bits u
        b = x.reshape(-1, 32)
        top = torch.frexp(b.abs().amax(1))[1].to(d) - 1  # floor of log2
        byte = torch.where(b.abs().amax(1) > 0, (top - 7 + 127).clamp(min=0), 0.0)
        scale = pow2(byte - 127)
        y = b.abs() / scale[:, None]
        step = pow2((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
        q = y / step
        low = q.floor()
        up = ((q - low) * 65536).floor() + u.reshape(-1, 32) >= 65536
        return (torch.sign(b) * (low + up) * step).flatten(), scale

    g = s["g"].to(d)
    m = h["beta1"] * state("m") + (1 - h["beta1"]) * g
    v = h["beta2"] * (state("v") ** 2 if eight else state("v")) + (1 - h["beta2"]) * g ** 2
    mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
    p = s["p"].to(d)
    decay = torch.zeros_like(p)
    decay[:s["nd"]] = s["wd"]
    p = p - h["lr"] * decay * p - h["lr"] * mh / (vh.sqrt() + h["eps"])
    out = dict(p=p, copy=p if s["copy"] is not None else None)
    if not eight:
        return dict(out, m=m, v=v)
    del g, mh, vh, decay
    bits = _philox(m.numel(), h["step"], h["seed"])
    (m, ms), (v, vs) = stored(m, bits & 0xFFFF), stored(v.sqrt(), bits >> 16)
    return dict(out, m=m, v=v, m_scale=ms, v_scale=vs)
