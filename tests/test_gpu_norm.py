"""GPU parity of the norms with the float64 oracle.

Bounds, in half steps e = 2^-24 of fp32: a sum of n terms in fp32, however it
is arranged, is within n e of the sum of magnitudes; results are a few more
roundings, then the rounding to the output's type (half a step: 2^-8 of a
bf16 value)."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob
from gpu_helpers import dev, host_bits

pytestmark = pytest.mark.gpu

E = ob.EPS32
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def make(rng, R, C, dtype, pad=0, offset=0.0, sd=1.0):
    """A [R, C] view with row stride C + pad, and its float64 values."""
    t = torch.from_numpy(rng.normal(offset, sd, (R, C + pad)).astype(np.float32)).to(dtype).cuda()[:, :C]
    return t, t.double().cpu().numpy()


def vec(rng, C, dtype, about):
    t = torch.from_numpy(rng.normal(about, 0.3, C).astype(np.float32)).to(dtype).cuda()
    return t, t.double().cpu().numpy()


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first {i}: got {got[i]!r} "
                             f"want {want[i]!r} tol {np.broadcast_to(tol, want.shape)[i]!r}")


def forward(R, C, xdt, ydt, kind, wdt=torch.float32, affine=True, bias=True, pad=0, ypad=0, offset=0.5,
            sd=2.0, eps=1e-5, seed=0):
    rng = np.random.default_rng(seed + R * 7 + C)
    x, xv = make(rng, R, C, xdt, pad, offset, sd)
    w, wv = vec(rng, C, wdt, 1.0) if affine else (None, None)
    b, bv = vec(rng, C, wdt, 0.0) if affine and bias else (None, None)
    ybuf = torch.full((R, C + ypad), float("nan"), dtype=ydt, device="cuda")
    y, mean, rstd = fq.layer_norm(x, w, b, eps=eps, kind=kind, y=ybuf[:, :C])
    torch.cuda.synchronize()
    rms = kind == fq.RMS_NORM
    want, wm, wr = ob.norm(xv, wv, bv, eps, rms)
    what = f"norm R={R} C={C} {xdt}->{ydt} kind={kind}"
    if ypad:
        assert torch.isnan(ybuf[:, C:]).all(), f"{what}: wrote past cols"
    n = C + 4
    em = np.zeros(R) if rms else n * E * np.abs(xv).mean(1) + E * np.abs(wm)
    d = xv - wm[:, None]
    var = (d * d).mean(1) + eps
    # the mean's error moves the sum of squares by C em^2 only
    er = 0.5 * ((n + 4) * E + em * em / var) + 4 * E
    near(rstd, wr, er * wr, what + " rstd")
    if rms:
        assert mean is None
    else:
        near(mean, wm, em, what + " mean")
    aw = np.ones(C) if wv is None else np.abs(wv)
    body = np.abs(d) * wr[:, None] * aw
    tol = body * (er[:, None] + 4 * E) + (em * wr)[:, None] * aw + E * (np.abs(want) + body)
    near(y, want, tol * (1 + HALF[ydt]) + HALF[ydt] * np.abs(want) + TINY[ydt], what + " y")


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
         (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)]
SIZES = [(1, 1), (1, 2), (3, 7), (2, 64), (5, 65), (4, 255), (3, 256), (2, 1000), (3, 1111), (9, 2048),
         (2, 4096), (2, 5120), (2, 5121), (2, 8192), (2, 13824), (1, 16385), (1, 40000), (300, 96)]
KINDS = [fq.LAYER_NORM, fq.RMS_NORM]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", SIZES)
def test_forward_sizes(R, C, kind):
    for xdt, ydt in TYPES:
        forward(R, C, xdt, ydt, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_forward_vectors_strides_and_offsets(kind):
    bf, f32 = torch.bfloat16, torch.float32
    for pad, ypad in ((0, 0), (8, 8), (3, 5), (1, 0)):
        forward(6, 512, bf, bf, kind, wdt=bf, pad=pad, ypad=ypad)
        forward(6, 511, f32, f32, kind, bias=False, pad=pad, ypad=ypad)
        forward(6, 520, bf, f32, kind, affine=False, pad=pad, ypad=ypad)
    forward(4, 2048, f32, f32, kind, offset=100.0, sd=1.0)  # a mean far above the spread
    forward(4, 2048, f32, f32, kind, sd=1e-18)              # squares below the normal range: eps rules
    forward(3, 300, f32, f32, kind, sd=1e15)


@pytest.mark.parametrize("kind", KINDS)
def test_forward_constant_rows_and_zero_eps(kind):
    x = torch.full((3, 96), 2.0, device="cuda")
    x[1] = 0.0
    y, mean, rstd = fq.layer_norm(x, eps=0.0625, kind=kind)
    torch.cuda.synchronize()
    want, _, wr = ob.norm(x.double().cpu().numpy(), None, None, 0.0625, kind == fq.RMS_NORM)
    assert np.allclose(y.cpu().numpy(), want, rtol=1e-6) and np.allclose(rstd.cpu().numpy(), wr, rtol=1e-6)
    # eps 0 on a zero row: rstd is infinite and the row is NaN, the others are not
    y, _, rstd = fq.layer_norm(x, eps=0.0, kind=kind)
    assert torch.isinf(rstd[1]) and torch.isnan(y[1]).all()


def test_forward_non_finite_rows_stay_alone():
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(5, 300, device="cuda").to(dt)
        ref = fq.layer_norm(x)[0]
        x2 = x.clone()
        x2[1, 17], x2[3, 299] = float("inf"), float("nan")
        y = fq.layer_norm(x2)[0]
        bad = torch.isnan(y).all(1).cpu().numpy()
        assert bad.tolist() == [False, True, False, True, False]
        assert torch.equal(y[[0, 2, 4]], ref[[0, 2, 4]])


def backward(R, C, xdt, dydt, kind, wdt=torch.float32, affine=True, pad=0, seed=0, scale=1e-3, inplace=False):
    rng = np.random.default_rng(seed + R * 5 + C)
    x, xv = make(rng, R, C, xdt, pad, 0.5, 2.0)
    dy, dyv = make(rng, R, C, dydt, pad, 0.0, scale)
    w, wv = vec(rng, C, wdt, 1.0) if affine else (None, None)
    rms = kind == fq.RMS_NORM
    _, mean, rstd = fq.layer_norm(x, w, kind=kind)
    mv = None if rms else mean.double().cpu().numpy()
    rv = rstd.double().cpu().numpy()
    dxb = torch.full((R, C + pad), float("nan"), dtype=xdt, device="cuda")
    dx = (dy if dydt == xdt else x) if inplace else dxb[:, :C]
    got = fq.layer_norm_grad(dy, x, w, mean, rstd, kind=kind, dx=dx)
    torch.cuda.synchronize()
    what = f"norm grad R={R} C={C} {xdt} dy {dydt} kind={kind}"
    if pad and not inplace:
        assert torch.isnan(dxb[:, C:]).all(), f"{what}: wrote past cols"
    want = ob.norm_grad(dyv, xv, wv, mv, rv, rms)
    xh = (xv - (0 if rms else mv[:, None])) * rv[:, None]
    t = dyv * (1 if wv is None else wv)
    atx, at = np.abs(t * xh).mean(1)[:, None], np.abs(t).mean(1)[:, None]
    tol = (6 * E * np.abs(t) + np.abs(xh) * (C + 12) * E * atx + (0 if rms else (C + 8) * E * at)
           + 4 * E * np.abs(want[0] / rv[:, None])) * rv[:, None]
    near(got[0], want[0], tol * (1 + HALF[xdt]) + HALF[xdt] * np.abs(want[0]) + TINY[xdt], what + " dx")
    near(got[1], want[1], (R + 8) * E * np.abs(dyv * xh).sum(0) + 2.0 ** -149, what + " dweight")
    near(got[2], want[2], (R + 8) * E * np.abs(dyv).sum(0) + 2.0 ** -149, what + " dbias")
    return got


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,C", SIZES + [(63, 40), (64, 40), (65, 40), (1000, 33), (2100, 72), (700, 2048)])
def test_backward_sizes(R, C, kind):
    for xdt, dydt in TYPES:
        backward(R, C, xdt, dydt, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_backward_vectors_strides_in_place(kind):
    bf, f32 = torch.bfloat16, torch.float32
    for pad in (0, 8, 3):
        backward(130, 512, bf, bf, kind, wdt=bf, pad=pad)
        backward(20, 511, f32, f32, kind, affine=False, pad=pad)
        backward(70, 520, f32, f32, kind, pad=pad, inplace=True)
        backward(70, 520, bf, f32, kind, pad=pad, inplace=True)
        backward(70, 513, bf, bf, kind, pad=pad, inplace=True)


def test_backward_matches_differences():
    """The whole gradient against central differences of the float64 forward."""
    rng = np.random.default_rng(1)
    R, C = 4, 24
    for kind in KINDS:
        rms = kind == fq.RMS_NORM
        x, xv = make(rng, R, C, torch.float32, 0, 0.3, 1.0)
        dy, dyv = make(rng, R, C, torch.float32)
        w, wv = vec(rng, C, torch.float32, 1.0)
        b, bv = vec(rng, C, torch.float32, 0.0)
        _, mean, rstd = fq.layer_norm(x, w, b, kind=kind)
        dx, dw, db = (t.double().cpu().numpy() for t in fq.layer_norm_grad(dy, x, w, mean, rstd, kind=kind))

        def loss(x, w, b):
            return (ob.norm(x, w, b, 1e-5, rms)[0] * dyv).sum()
        h = 1e-5
        for i in range(R):
            for j in range(0, C, 5):
                e = np.zeros_like(xv)
                e[i, j] = h
                d = (loss(xv + e, wv, bv) - loss(xv - e, wv, bv)) / (2 * h)
                assert abs(d - dx[i, j]) < 1e-4 * (1 + abs(d))
        for j in range(C):
            e = np.zeros(C)
            e[j] = h
            assert abs((loss(xv, wv + e, bv) - loss(xv, wv - e, bv)) / (2 * h) - dw[j]) < 1e-4
            assert abs((loss(xv, wv, bv + e) - loss(xv, wv, bv - e)) / (2 * h) - db[j]) < 1e-4


def test_backward_parts_on_their_own_and_repeatable():
    x, dy = torch.randn(2, 500, 320, device="cuda")
    w = torch.randn(320, device="cuda")
    _, mean, rstd = fq.layer_norm(x, w)
    full = fq.layer_norm_grad(dy, x, w, mean, rstd)
    again = fq.layer_norm_grad(dy, x, w, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(full, again))
    dx, dw, db = fq.layer_norm_grad(dy, x, w, mean, rstd, want_weight=False, want_bias=False)
    assert torch.equal(dx, full[0]) and dw is None and db is None
    _, dw, db = fq.layer_norm_grad(dy, x, w, mean, rstd, want_bias=False)
    assert torch.equal(dw, full[1]) and db is None
    _, dw, db = fq.layer_norm_grad(dy, x, w, mean, rstd, want_weight=False)
    assert dw is None and torch.equal(db, full[2])


def test_backward_refuses_broadcast_rows_and_short_workspaces():
    x = torch.randn(8, 64, device="cuda")
    _, mean, rstd = fq.layer_norm(x)
    with pytest.raises(fq.Fp4qError, match="row stride"):
        fq.layer_norm_grad(torch.ones(1, 64, device="cuda").expand(8, 64), x, None, mean, rstd)
    with pytest.raises(fq.Fp4qError, match="workspace"):
        fq.layer_norm_grad(x, x, None, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        fq.layer_norm_grad(x[:4], x, None, mean, rstd)


def test_other_stream_and_graph_replays():
    x, dy = torch.randn(2, 700, 520, device="cuda").bfloat16()
    w, b = torch.randn(2, 520, device="cuda")

    def step(stream=None):
        y, mean, rstd = fq.layer_norm(x, w, b, stream=stream)
        return (y, mean, rstd, *fq.layer_norm_grad(dy, x, w, mean, rstd, stream=stream))
    want = [host_bits(t) for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(np.array_equal(host_bits(a), c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host_bits(a), c) for a, c in zip(out, want))
        step()


@pytest.mark.parametrize("C", [5, 300, 1500, 20000])
def test_rms_rows_with_an_infinity_and_overflowing_squares(C):
    """RMS norm: the sum of squares is infinite, so rstd is 0, the infinity
    itself NaN and the row's finite elements the bias; a NaN takes the row.
    Squares beyond fp32 act alike in either kind, with no NaN."""
    w, b = torch.randn(2, C, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(5, C, device="cuda").to(dt)
        ref = fq.layer_norm(x, w, b, kind=fq.RMS_NORM)[0]
        x2 = x.clone()
        x2[1, C // 2], x2[3, C - 1] = float("-inf"), float("nan")
        y, _, rstd = fq.layer_norm(x2, w, b, kind=fq.RMS_NORM)
        want = b.to(dt).clone()
        want[C // 2] = float("nan")
        assert torch.equal(y[1].isnan(), want.isnan())
        assert torch.equal(y[1].nan_to_num(), want.nan_to_num()) and rstd[1] == 0
        assert y[3].isnan().all() and rstd[3].isnan()
        assert torch.equal(y[[0, 2, 4]], ref[[0, 2, 4]])
        for kind in KINDS:
            x2 = x.clone()
            x2[2, 0] = 1e25
            y, _, rstd = fq.layer_norm(x2, w, b, kind=kind)
            assert rstd[2] == 0 and torch.equal(y[2], b.to(dt))
            assert torch.isfinite(y).all()
