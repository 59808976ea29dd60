"""GPU parity of the residual norms with the float64 oracle.

Bounds, in half steps e = 2^-24 of fp32: a sum of n terms in fp32, however it
is arranged, is within n e of the sum of magnitudes; an error of an operand
goes through the formula's derivative; results are a few more roundings, then
the rounding to the output's type (half a step: 2^-8 of a bf16 value, 2^-24 of
an fp32 one)."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob
from gpu_helpers import host_bits

pytestmark = pytest.mark.gpu

E = ob.EPS32
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, F32: 2.0 ** -149}
LAYER, RMS, NONE = fq.LAYER_NORM, fq.RMS_NORM, fq.NO_NORM


def make(rng, R, C, dtype, pad=0, offset=0.0, sd=1.0):
    """A [R, C] view with row stride C + pad, and its float64 values."""
    t = torch.from_numpy(rng.normal(offset, sd, (R, C + pad)).astype(np.float32)).to(dtype).cuda()[:, :C]
    return t, t.double().cpu().numpy()


def vec(rng, C, dtype, about):
    t = torch.from_numpy(rng.normal(about, 0.3, C).astype(np.float32)).to(dtype).cuda()
    return t, t.double().cpu().numpy()


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, f"{what}: shape {got.shape}, not {want.shape}"
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} tol {np.broadcast_to(tol, want.shape)[i]!r}")


def stored(tol, want, dtype):
    """Bound of a value with error tol that is rounded to dtype."""
    return tol * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) + TINY[dtype]


def one(v, C):
    return np.ones(C) if v is None else v


def norm_bound(v, tv, mean, rstd, w, y, rms, eps):
    """Bounds of (mean, rstd, y) of a norm whose input v has error tv."""
    C = v.shape[1]
    n = C + 4
    em = np.zeros(len(v)) if rms else n * E * np.abs(v).mean(1) + tv.mean(1) + E * np.abs(mean)
    d = v - (0 if rms else mean[:, None])
    var = (d * d).mean(1) + eps
    move = tv + em[:, None]  # of each centred element; the mean's part leaves the first order
    er = 0.5 * ((n + 4) * E + (2 * (np.abs(d) * tv).mean(1) + (move * move).mean(1)) / var) + 4 * E
    aw = np.abs(one(w, C))
    body = np.abs(d) * rstd[:, None] * aw
    ty = body * (er[:, None] + 4 * E) + move * rstd[:, None] * aw + E * (np.abs(y) + body)
    return em, er * rstd, ty


class Case:
    """Operands of a call, its keyword arguments and float64 values."""

    def __init__(self, R, C, xdt=BF, bdt=BF, post=LAYER, kind=LAYER, gates=0, wdt=F32, affine=True, bias=True,
                 pad=0, xs=1.0, bs=1.0, offset=0.5, sd=2.0, eps=1e-5, seed=0, gdt=None):
        rng = np.random.default_rng(seed + R * 7 + C)
        self.R, self.C, self.post, self.kind, self.rms, self.eps = R, C, post, kind, kind == RMS, eps
        self.xs, self.bs, self.pad, self.rng = xs, bs, pad, rng
        self.x, self.xv = make(rng, R, C, xdt, pad, offset, sd)
        self.b, self.bv = make(rng, R, C, bdt, pad, -0.25, sd)
        none = (None, None)
        self.w, self.wv = vec(rng, C, wdt, 1.0) if affine else none
        self.c, self.cv = vec(rng, C, wdt, 0.0) if affine and bias else none
        self.pw, self.pwv = vec(rng, C, wdt, 1.0) if affine and post != NONE else none
        self.pc, self.pcv = vec(rng, C, wdt, 0.0) if affine and bias and post != NONE else none
        self.each = min(gates, R) if gates else R  # rows of a gate
        self.g, self.gv = make(rng, -(-R // self.each), C, gdt or bdt, pad, 0.5, 0.5) if gates else none
        self.kw = dict(kind=kind, post_kind=post, post_weight=self.pw, post_bias=self.pc, gate=self.g,
                       gate_rows=self.each if gates else None, x_scale=xs, branch_scale=bs)
        self.what = f"R={R} C={C} {xdt} {bdt} post={post} kind={kind} gates={gates} pad={pad}"

    def forward(self, **kw):
        return fq.residual_norm(self.x, self.b, self.w, self.c, eps=self.eps, **self.kw, **kw)

    def check_forward(self, ydt):
        R, C, pad = self.R, self.C, self.pad
        xb = torch.full((R, C + pad), float("nan"), dtype=self.x.dtype, device="cuda")
        yb = torch.full((R, C + pad), float("nan"), dtype=ydt, device="cuda")
        xo, y, stats = self.forward(x_out=xb[:, :C], y=yb[:, :C])
        torch.cuda.synchronize()
        if pad:
            assert xb[:, C:].isnan().all() and yb[:, C:].isnan().all(), f"{self.what}: wrote past cols"
        wx, wy, (pm, pr, m, r) = ob.residual_norm(self.xv, self.bv, self.post, self.pwv, self.pcv, self.gv, self.each,
                                                  self.xs, self.bs, self.rms, self.wv, self.cv, self.eps)
        bounds = []
        n, tn = self.bv, np.zeros_like(self.bv)
        if self.post != NONE:
            n = ob.norm(self.bv, self.pwv, self.pcv, self.eps, self.post == RMS)[0]
            tm, tr, tn = norm_bound(self.bv, tn, pm, pr, self.pwv, n, self.post == RMS, self.eps)
            tn = tn + 3 * E * (np.abs(n) + (0 if self.pcv is None else np.abs(self.pcv)))
            bounds += [(stats[0], pm, tm, "post_mean"), (stats[1], pr, tr, "post_rstd")]
        f = self.bs * ob.group_rows(self.gv, R, self.each)
        tx = np.abs(f) * tn + 4 * E * (np.abs(self.xs * self.xv) + np.abs(f * n)) + E * np.abs(wx)
        tm, tr, ty = norm_bound(wx, tx, m, r, self.wv, wy, self.rms, self.eps)
        bounds += [(stats[2], m, tm, "mean"), (stats[3], r, tr, "rstd")]
        for got, want, tol, name in bounds:
            if "mean" in name and (self.post if name == "post_mean" else self.kind) == RMS:
                assert got is None
            else:
                near(got, want, tol, f"{self.what} {name}")
        if self.post == NONE:
            assert stats[0] is None and stats[1] is None
        near(xo, wx, stored(tx, wx, self.x.dtype), f"{self.what} x_out")
        near(y, wy, stored(ty, wy, ydt), f"{self.what} y {ydt}")
        return xo, y, stats

    def gradients(self, dydt, stream_grad=True, scale=1e-3, inplace=False, **kw):
        """Runs forward and backward; returns the gradients by name with their
        oracle values and bounds."""
        R, C, pad = self.R, self.C, self.pad
        xo, _, stats = self.forward()
        dy, dyv = make(self.rng, R, C, dydt, pad, 0.0, scale)
        dxo, dxov = make(self.rng, R, C, self.x.dtype, pad, 0.0, scale) if stream_grad else (None, None)
        xov = xo.double().cpu().numpy()
        sv = [None if s is None else s.double().cpu().numpy() for s in stats]
        dxb = torch.full((R, C + pad), float("nan"), dtype=self.x.dtype, device="cuda")
        dbb = torch.full((R, C + pad), float("nan"), dtype=self.b.dtype, device="cuda")
        dx, db = dxb[:, :C], dbb[:, :C]
        if inplace:
            dx, db = dxo, self.b
        names = ("dx", "dbranch", "dweight", "dbias", "dpost_weight", "dpost_bias", "dgate")
        post = self.post != NONE
        got = dict(zip(names, fq.residual_norm_grad(dy, dxo, xo, self.b, stats, self.w, dx=dx, dbranch=db,
                                                    **{**dict(want_post_weight=post, want_post_bias=post), **self.kw,
                                                       **kw})))
        torch.cuda.synchronize()
        if pad and not inplace:
            assert dxb[:, C:].isnan().all() and dbb[:, C:].isnan().all(), f"{self.what}: wrote past cols"
        want = ob.residual_norm_grad(dyv, dxov, xov, self.bv, sv, self.post, self.pwv, self.pcv, self.gv, self.each,
                                     self.xs, self.bs, self.rms, self.wv)
        return got, want, self.grad_bounds(dyv, xov, sv, want)

    def grad_bounds(self, dyv, xov, sv, want):
        R, C = self.R, self.C
        pm, pr, m, r = (None if s is None else s[:, None] for s in sv)

        def back(t, tt, h, th, mine, rstd, layer):
            """Bound of rstd (t - mean t - h mean(t h)) for t, h with errors tt, th."""
            ath, at = np.abs(t * h).mean(1, keepdims=True), np.abs(t).mean(1, keepdims=True)
            t1 = (C + 12) * E * ath + (tt * np.abs(h) + np.abs(t) * th).mean(1, keepdims=True)
            t0 = (C + 8) * E * at + tt.mean(1, keepdims=True) if layer else 0.0
            body = np.abs(t) + np.abs(h) * ath + (at if layer else 0.0)
            return rstd * (tt + np.abs(h) * t1 + th * ath + t0 + 5 * E * body) + 2 * E * np.abs(mine)
        xh = (xov - (0 if self.rms else m)) * r
        t = dyv * one(self.wv, C)
        D = want["dx"] / self.xs
        tD = back(t, E * np.abs(t), xh, 2 * E * np.abs(xh), D, r, not self.rms) + 2 * E * np.abs(D)
        tol = dict(dx=np.abs(self.xs) * tD + 2 * E * np.abs(want["dx"]),
                   dweight=(R + 8) * E * np.abs(dyv * xh).sum(0), dbias=(R + 8) * E * np.abs(dyv).sum(0))
        f = self.bs * ob.group_rows(self.gv, R, self.each) * np.ones((R, C))
        h = self.bv if self.post == NONE else (self.bv - (0 if self.post == RMS else pm)) * pr
        th = np.zeros_like(h) if self.post == NONE else 2 * E * np.abs(h)
        u = f * D * one(self.pwv, C)
        tu = np.abs(f * one(self.pwv, C)) * tD + 5 * E * np.abs(u)
        if self.post == NONE:
            tol["dbranch"] = tu
        else:
            tol["dbranch"] = back(u, tu, h, th, want["dbranch"], pr, self.post == LAYER)
            # sums of D h and D over a gate's rows, then over the gates
            s1, s2 = np.abs(D * h), np.abs(D)
            t1, t2 = tD * np.abs(h) + np.abs(D) * th, tD
            tol["dpost_weight"] = (np.abs(f) * (t1 + (R + 12) * E * s1)).sum(0)
            tol["dpost_bias"] = (np.abs(f) * (t2 + (R + 12) * E * s2)).sum(0)
        if self.gv is not None:
            aw, ac = np.abs(one(self.pwv, C)), 0.0 if self.pcv is None else np.abs(self.pcv)
            parts = (aw * (tD * np.abs(h) + np.abs(D) * th + (self.each + 12) * E * np.abs(D * h))
                     + ac * (tD + (self.each + 12) * E * np.abs(D)))
            tol["dgate"] = np.stack([np.abs(self.bs) * parts[i:i + self.each].sum(0)
                                     for i in range(0, R, self.each)])
        return tol

    def check_backward(self, dydt, **kw):
        got, want, tol = self.gradients(dydt, **kw)
        for name, w in want.items():
            g = got[name]
            near(g, w, stored(tol[name], w, g.dtype), f"{self.what} dy {dydt} {name}")
        for name, g in got.items():
            assert (g is None) == (name not in want), name
        return got


TYPES = [(BF, BF, BF), (F32, F32, F32), (F32, BF, BF), (BF, F32, F32)]  # x, branch, y
SIZES = [(1, 1), (1, 2), (3, 7), (2, 8), (2, 64), (5, 65), (4, 255), (3, 256), (4, 512), (2, 1000), (3, 1111),
         (9, 2048), (2, 4096), (2, 5121), (2, 8192), (2, 8200), (2, 13824), (1, 16385), (300, 96)]
KINDS = [(LAYER, LAYER), (RMS, RMS), (NONE, LAYER), (LAYER, RMS)]  # post, kind


@pytest.mark.parametrize("post,kind", KINDS)
@pytest.mark.parametrize("R,C", SIZES)
def test_forward_sizes(R, C, post, kind):
    for i, (xdt, bdt, ydt) in enumerate(TYPES):
        Case(R, C, xdt, bdt, post, kind, gates=(0, R, 1, 2)[i], bs=(1.0, 0.22)[i % 2]).check_forward(ydt)


@pytest.mark.parametrize("post,kind", KINDS)
def test_forward_vectors_strides_gates_and_offsets(post, kind):
    for pad in (0, 8, 3):
        Case(6, 512, BF, BF, post, kind, wdt=BF, pad=pad, gates=4, xs=0.5).check_forward(BF)
        Case(6, 511, F32, F32, post, kind, bias=False, pad=pad, gates=5, gdt=BF).check_forward(F32)
        Case(6, 520, BF, F32, post, kind, affine=False, pad=pad, gates=6).check_forward(F32)
    Case(4, 2048, F32, F32, post, kind, offset=100.0, sd=1.0, bs=-2.0).check_forward(F32)
    Case(4, 2048, F32, F32, post, kind, sd=1e-18).check_forward(F32)  # squares below the normal range: eps rules
    Case(3, 300, F32, F32, post, kind, sd=1e15, xs=-1.0).check_forward(F32)


@pytest.mark.parametrize("C", [32, 96, 1056, 2048, 5152, 13824, 16416])
def test_codes_are_the_quantised_y(C):
    """Bit for bit fp4q_quantize of y in fp32, a block with an Inf or NaN among
    them."""
    for xdt, bdt in ((BF, BF), (F32, BF)):
        c = Case(7, C, xdt, bdt, RMS, LAYER, gates=3)
        c.x[2, C // 2] = float("nan")
        c.x[4, C - 1] = 3e38 if xdt == F32 else float("inf")
        c.b[5, 0] = float("inf")
        xo, y, stats = c.forward(out_dtype=F32)
        xq, (codes, scales), qstats = c.forward(quantize=True)
        wc, ws = fq.quantize(y, 32)
        assert torch.equal(codes, wc) and torch.equal(scales, ws)
        same = [(a, b) for a, b in zip((xo, *stats), (xq, *qstats)) if a is not None]
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in same)
    with pytest.raises(ValueError, match="32"):
        fq.residual_norm(c.x[:, :C - 8], c.b[:, :C - 8], quantize=True)


@pytest.mark.parametrize("C", [5, 300, 2048, 13824, 20000])
def test_rows_stay_alone(C):
    """An Inf or NaN anywhere in x, the branch or a gate's row reaches its own
    rows only; x_out may be x."""
    for dt in (BF, F32):
        c = Case(9, C, dt, dt, LAYER, RMS, gates=1)
        ref = c.forward()
        for t, i in ((c.x, 1), (c.b, 4), (c.g, 6)):
            t[i, C // 2] = float("nan")
        c.x[8, C - 1] = float("inf")
        xo, y, stats = c.forward()
        keep = [0, 2, 3, 5, 7]
        for a, b in ((xo, ref[0]), (y, ref[1]), *zip(stats[:2] + stats[3:], ref[2][:2] + ref[2][3:])):
            assert torch.equal(a[keep], b[keep])
        assert y[[1, 4, 6]].isnan().all() and xo[4].isnan().all() and int(xo[1].isnan().sum()) == 1
        into = c.x.clone()
        c.x = into
        x2, y2, _ = c.forward(x_out=into)
        assert x2 is into and torch.equal(x2.nan_to_num(5.0), xo.nan_to_num(5.0))
        assert torch.equal(y2.nan_to_num(5.0), y.nan_to_num(5.0))


@pytest.mark.parametrize("post,kind", KINDS)
@pytest.mark.parametrize("R,C", SIZES + [(63, 40), (65, 40), (1000, 33), (1100, 600), (2100, 72), (700, 2048)])
def test_backward_sizes(R, C, post, kind):
    for i, (xdt, bdt, dydt) in enumerate(TYPES):
        gates = (0, R, 1 if R * C < 100000 else 40, max(1, R // 3))[i]
        Case(R, C, xdt, bdt, post, kind, gates=gates, bs=(1.0, 0.22)[i % 2]).check_backward(dydt)


@pytest.mark.parametrize("gates", [1, 2, 3, 7, 16, 31, 100, 129, 499, 500, 1000])
def test_backward_gates_of_any_length(gates):
    """Groups shorter and longer than what a workgroup takes, the last one
    short, in every way that a row is held."""
    for C in (6, 72, 520, 1030, 8200):
        R = 500 if C < 8200 else 60
        Case(R, C, F32, F32, LAYER, RMS, gates=gates, gdt=BF).check_backward(F32)
    Case(500, 136, BF, BF, NONE, LAYER, gates=gates, xs=0.5).check_backward(BF)
    Case(1500, 1000, BF, BF, RMS, LAYER, gates=gates, xs=0.5).check_backward(BF)


@pytest.mark.parametrize("post,kind", KINDS)
def test_backward_vectors_strides_in_place(post, kind):
    for pad in (0, 8, 3):
        Case(130, 512, BF, BF, post, kind, wdt=BF, pad=pad, gates=50).check_backward(BF)
        Case(20, 511, F32, F32, post, kind, affine=False, pad=pad).check_backward(F32, stream_grad=False)
        Case(70, 520, F32, BF, post, kind, pad=pad, gates=9).check_backward(F32, inplace=True)
        Case(70, 513, BF, F32, post, kind, pad=pad).check_backward(BF, inplace=True)
        Case(20, 8209, BF, BF, post, kind, pad=pad, gates=3).check_backward(BF, inplace=True)
        Case(9, 16400, F32, F32, post, kind, pad=pad, gates=2).check_backward(F32, inplace=True)
        Case(30, 2056, BF, BF, post, kind, pad=pad, bias=False).check_backward(F32, stream_grad=False)


def test_backward_matches_differences():
    """The gradients against central differences of the float64 forward."""
    c = Case(6, 24, F32, F32, LAYER, LAYER, gates=2, bs=0.4, sd=1.0)
    got, _, _ = c.gradients(F32, scale=1.0)
    d = Case(6, 24, F32, F32, LAYER, LAYER, gates=2, bs=0.4, sd=1.0)
    _, dyv = make(d.rng, 6, 24, F32, 0, 0.0, 1.0)
    _, dxov = make(d.rng, 6, 24, F32, 0, 0.0, 1.0)
    base = dict(x=c.xv, b=c.bv, pw=c.pwv, pc=c.pcv, g=c.gv, w=c.wv, c=c.cv)

    def loss(**kw):
        v = {**base, **kw}
        xo, y, _ = ob.residual_norm(v["x"], v["b"], 0, v["pw"], v["pc"], v["g"], 2, 1.0, 0.4, False, v["w"], v["c"],
                                    1e-5)
        return (y * dyv).sum() + (xo * dxov).sum()
    for name, arg in (("dx", "x"), ("dbranch", "b"), ("dweight", "w"), ("dbias", "c"), ("dpost_weight", "pw"),
                      ("dpost_bias", "pc"), ("dgate", "g")):
        flat = got[name].double().cpu().numpy().ravel()
        for i in range(0, flat.size, 5):
            e = np.zeros(flat.size)
            e[i] = 1e-5
            e = e.reshape(base[arg].shape)
            diff = (loss(**{arg: base[arg] + e}) - loss(**{arg: base[arg] - e})) / 2e-5
            assert abs(diff - flat[i]) < 2e-4 * (1 + abs(diff)), (name, i)


@pytest.mark.parametrize("C", [5, 96, 1000, 2048, 13824])
def test_backward_parts_on_their_own_and_repeatable(C):
    c = Case(90, C, BF, BF, RMS, LAYER, gates=40)
    xo, _, stats = c.forward()
    dy, dxo = (make(c.rng, 90, C, BF, 0, 0.0, 1e-3)[0] for _ in range(2))

    def grad(**kw):
        return fq.residual_norm_grad(dy, dxo, xo, c.b, stats, c.w, **c.kw, **kw)
    full = grad()
    assert all(torch.equal(a, b) for a, b in zip(full, grad()))
    wants = ("want_weight", "want_bias", "want_post_weight", "want_post_bias", "want_gate")
    for k in range(5):
        got = grad(**{w: i == k for i, w in enumerate(wants)})
        for i, (a, b) in enumerate(zip(got, full)):
            assert torch.equal(a, b) if i < 2 or i == k + 2 else a is None
    none = grad(**{w: False for w in wants})
    assert torch.equal(none[0], full[0]) and torch.equal(none[1], full[1]) and none[2:] == (None,) * 5
    # no norm behind the block, no gradient of the gate: the branch is not read
    kw = {**c.kw, "post_kind": NONE, "post_weight": None, "post_bias": None}
    a = fq.residual_norm_grad(dy, dxo, xo, c.b, (None, None, *stats[2:]), c.w, want_gate=False, **kw)
    b = fq.residual_norm_grad(dy, dxo, xo, None, (None, None, *stats[2:]), c.w, want_gate=False, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a[:4], b[:4]))


@pytest.mark.parametrize("C", [7, 300, 2048, 8200])
def test_backward_non_finite_rows_stay_alone(C):
    c = Case(20, C, F32, F32, LAYER, LAYER, gates=1)
    xo, _, stats = c.forward()
    dy, dxo = (make(c.rng, 20, C, F32, 0, 0.0, 1e-3)[0] for _ in range(2))
    run = lambda: fq.residual_norm_grad(dy, dxo, xo, c.b, stats, c.w, **c.kw)  # noqa: E731
    ref = run()
    dy[3, C // 2], dxo[9, 0] = float("nan"), float("inf")
    got = run()
    keep = [i for i in range(20) if i not in (3, 9)]
    for i in (0, 1, 6):  # dx, dbranch, and dgate: a gate per row
        assert torch.equal(got[i][keep], ref[i][keep])
    assert got[0][3].isnan().all() and torch.isinf(got[0][9, 0])


def test_backward_refuses_short_workspaces_and_broadcast_rows():
    c = Case(8, 64, gates=2)
    xo, _, stats = c.forward()
    with pytest.raises(fq.Fp4qError, match="workspace"):
        fq.residual_norm_grad(xo, xo, xo, c.b, stats, c.w, **c.kw,
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fq.Fp4qError, match="row stride"):
        fq.residual_norm_grad(xo[:1].expand(8, 64), xo, xo, c.b, stats, c.w, **c.kw)
    with pytest.raises(fq.Fp4qError, match="row stride"):
        c.kw["gate"] = c.g[:1].expand(4, 64)
        c.forward()


@pytest.mark.parametrize("C", [520, 2048])
def test_other_stream_and_graph_replays(C):
    c = Case(700, C, BF, BF, RMS, LAYER, gates=300)
    dy, dxo = (make(c.rng, 700, C, BF, 0, 0.0, 1e-3)[0] for _ in range(2))

    def step(stream=None):
        xo, y, stats = c.forward(stream=stream)
        q = c.forward(stream=stream, quantize=True)[1] if C % 32 == 0 else ()
        back = fq.residual_norm_grad(dy, dxo, xo, c.b, stats, c.w, **c.kw, stream=stream)
        return [t for t in (xo, y, *stats, *q, *back) if t is not None]
    want = [host_bits(t) for t in step()]
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(2):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                a @ a
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(np.array_equal(host_bits(t), w) for t, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host_bits(t), w) for t, w in zip(out, want))
        step()


@pytest.mark.parametrize("C", [5, 300, 1000, 2048, 9000, 20000])
def test_overflowing_squares(C):
    """Finite elements whose squares overflow fp32 make the norm's rstd 0 and its
    output the bias, in front of the sum as behind it, and leave other rows alone."""
    for post, kind in ((LAYER, LAYER), (RMS, RMS)):
        c = Case(5, C, F32, F32, post, kind)
        ref = c.forward()
        c.b[1, C // 2], c.x[3, 0] = 1e25, -1e25
        xo, y, (_, pr, _, r) = c.forward()
        assert pr[1] == 0 and r[3] == 0 and xo.isfinite().all() and y.isfinite().all()
        assert torch.equal(xo[1], c.x[1] + c.pc) and torch.equal(y[3], c.c)
        keep = [0, 2, 4]
        assert torch.equal(xo[keep], ref[0][keep]) and torch.equal(y[keep], ref[1][keep])


def test_offsets_beyond_32_bits():
    """The last rows of operands of more than 2^31 elements: the same bits as
    from a call on them alone."""
    R, C, last = 270001, 8192, 5
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def big():
        t = torch.zeros(R, C, dtype=BF, device="cuda")
        t[-last:] = torch.randn(last, C, generator=g, device="cuda").to(BF)
        return t
    x, b, dy, dxo = (big() for _ in range(4))
    w = torch.rand(C, generator=g, device="cuda") + 0.5
    kw = dict(kind=RMS, post_kind=RMS, post_weight=w)
    xo, y, stats = fq.residual_norm(x, b, w, **kw)
    few = [t[-last:].contiguous() for t in (x, b, dy, dxo)]
    xo2, y2, stats2 = fq.residual_norm(few[0], few[1], w, **kw)
    assert torch.equal(xo[-last:], xo2) and torch.equal(y[-last:], y2) and torch.equal(stats[3][-last:], stats2[3])
    assert not xo[:-last].any() and not y[:-last].any()
    full = fq.residual_norm_grad(dy, dxo, xo, b, stats, w, **kw)
    part = fq.residual_norm_grad(few[2], few[3], xo2, few[1], stats2, w, **kw)
    assert torch.equal(full[0][-last:], part[0]) and torch.equal(full[1][-last:], part[1])
    assert not full[0][:-last].any() and not full[1][:-last].any()
    # the sums of the few rows that are not zero, in another order: 2 roundings a row
    for a, e in zip(full[2:5], part[2:5]):
        assert torch.allclose(a, e, rtol=0, atol=10 * E * float(e.abs().max()) * last)
    _, (codes, scales), _ = fq.residual_norm(x, b, w, quantize=True, **kw)
    wc, ws = fq.residual_norm(few[0], few[1], w, quantize=True, **kw)[1]
    assert torch.equal(codes[-last:], wc) and torch.equal(scales[-last:], ws)


def test_two_calls_at_once():
    """Calls on two streams have workspaces of their own."""
    cases = [Case(900, C, BF, BF, RMS, LAYER, gates=g) for C, g in ((520, 300), (2048, 7))]
    work = []
    for c in cases:
        xo, _, stats = c.forward()
        dy, dxo = (make(c.rng, c.R, c.C, BF, 0, 0.0, 1e-3)[0] for _ in range(2))
        work.append((c, dy, dxo, xo, stats))

    def grad(c, dy, dxo, xo, stats):
        return fq.residual_norm_grad(dy, dxo, xo, c.b, stats, c.w, **c.kw)
    want = [[host_bits(t) for t in grad(*w)] for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        got = []
        for s, w in zip(streams, work):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(grad(*w))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(np.array_equal(host_bits(t), e) for t, e in zip(a, b))


@pytest.mark.parametrize("C", [513, 1025, 1540, 2055, 3001, 3600, 4100, 4608, 5125, 6144, 6145, 7170, 8185])
def test_every_number_of_waves(C):
    """Rows of every number of waves, teams that share a workgroup among them,
    rows that do not divide among the teams, with and without a gate per row."""
    for i, R in enumerate((3, 13, 45)):
        Case(R, C, BF, F32, LAYER, RMS, gates=(0, 1, 4)[i]).check_backward(BF)
        Case(R, C, F32, BF, RMS, LAYER, gates=(1, R, 0)[i]).check_backward(F32, inplace=i == 1)
        Case(R, C, BF, BF, LAYER, LAYER, gates=(1, 0, 4)[i]).check_forward(F32)


def test_many_short_rows():
    """Rows of one or two chunks per lane that a wave holds alone."""
    for C in (96, 520, 600, 1000, 1024):
        c = Case(1100, C, BF, BF, RMS, LAYER, gates=300)
        c.check_forward(BF)
        if C % 32 == 0:
            y, (codes, scales) = c.forward(out_dtype=F32)[1], c.forward(quantize=True)[1]
            wc, ws = fq.quantize(y, 32)
            assert torch.equal(codes, wc) and torch.equal(scales, ws)
