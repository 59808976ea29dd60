"""GPU parity of the gated feed-forward calls with the float64 oracle.

Bounds: a product is within 1e-5 S of its exact value (S the sum of absolute
products), as for fp4q_gemm; the activation's sigmoid within (4 |z| + 16) half
steps of fp32, relative (the exponent's argument is rounded a few times, and
its absolute error is the result's relative one); an output is then rounded
once to bf16, so it has to lie between the roundings of the ends of its
interval."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from mxfp4_block_scaled_fp4q_amd import inputs
from oracle import blocks as ob
from gpu_helpers import GEMM_REL, check_gemm_bf16, dev, dev_bf16, host_bits

pytestmark = pytest.mark.gpu

NAN16 = 0x7FC1  # what output buffers hold before a call


def bracket(got_bits, want, tol, orc, what):
    lo = orc.bf16_to_f64(orc.round_bf16(want - tol))
    hi = orc.bf16_to_f64(orc.round_bf16(want + tol))
    v = orc.bf16_to_f64(got_bits)
    bad = ~((v >= lo) & (v <= hi))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} outside; first {i}: got {v[i]!r} bracket "
                             f"[{lo[i]!r}, {hi[i]!r}] want {want[i]!r}")


def act_tol(z):
    return (4 * np.abs(z) + 16) * ob.EPS32


def filled(M, F, ld):
    t = torch.full((M, ld), NAN16, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    return t, t[:, :F]


def quant(orc, rows, K, seed, sd):
    x = inputs.with_outliers(inputs.normal((rows, K), seed) * np.float32(sd), seed + 1,
                             max(1, rows * K // 100), 8.0)
    return orc.quantize(x, 32)


def forward_check(orc, x, g, u, act, save, pad=0, rows=None):
    (xc, xs), (gc, gs), (uc, us) = x, g, u
    M, F = xc.shape[0], gc.shape[0]
    bufs = [filled(M, F, F + pad) for _ in range(3)]
    h, gate, up = (b[1] for b in bufs)
    kw = dict(gate=gate, up=up) if save else {}
    fq.gemm_gated(dev(xc), dev(xs), dev(gc), dev(gs), dev(uc), dev(us), act=act, h=h, **kw)
    torch.cuda.synchronize()
    sel = np.arange(M) if rows is None else rows
    G, Sg = orc.gemm_dense(xc, xs, gc, gs, rows=sel)
    U, Su = orc.gemm_dense(xc, xs, uc, us, rows=sel)
    s, z, dz = ob.act_parts(G, act)
    eg, eu = GEMM_REL * Sg, GEMM_REL * Su
    # |act'| <= 1.13 for both; the activation of a value eg away
    tol = 1.2 * eg * (np.abs(U) + eu) + np.abs(G * s) * eu + np.abs(G * s * U) * act_tol(z)
    what = f"gated M={M} F={F} K={2 * xc.shape[1]} act={act} save={save}"
    for t, _ in bufs:
        assert (host_bits(t)[:, F:] == NAN16).all(), f"{what}: wrote past F"
    bracket(host_bits(h)[sel], ob.gated(G, U, act), tol, orc, what + " h")
    if save:
        check_gemm_bf16(host_bits(gate)[sel], G, Sg, orc, what + " gate")
        check_gemm_bf16(host_bits(up)[sel], U, Su, orc, what + " up")
    return h, gate, up


SIZES = [(1, 1, 64), (1, 33, 128), (3, 129, 192), (17, 200, 320), (32, 64, 256), (33, 48, 1024),
         (65, 130, 2112), (130, 257, 960), (257, 129, 384), (300, 200, 256), (129, 769, 64)]


@pytest.mark.parametrize("act", [fq.SILU, fq.GELU])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_forward(orc, M, F, K, act):
    x, g, u = quant(orc, M, K, M, 1.0), quant(orc, F, K, F + 7, 0.05), quant(orc, F, K, F + 9, 0.05)
    forward_check(orc, x, g, u, act, save=True, pad=8)
    forward_check(orc, x, g, u, act, save=False, pad=3)


@pytest.mark.parametrize("M", [1, 2, 16, 31, 64, 128, 200, 512, 1100])
def test_forward_row_counts_agree_and_match(orc, M):
    """The projections of a 2048-wide block for growing numbers of rows."""
    K, F = 2048, 1408
    x, g, u = quant(orc, M, K, 5, 1.0), quant(orc, F, K, 6, 0.02), quant(orc, F, K, 8, 0.02)
    rows = np.unique(np.linspace(0, M - 1, 9).astype(int))
    forward_check(orc, x, g, u, fq.SILU, save=True, rows=rows)


# 128-row tiles, 256-row tiles and 256 x 256 tiles, with and without a half K step
TILED = [(250, 1500, 448), (1100, 800, 1152), (1100, 2990, 192), (900, 3900, 1664), (2100, 4100, 320),
         (2050, 4000, 2176)]


def some_rows(M):
    return np.unique(np.r_[0, 1, M // 2, M - 1, np.linspace(0, M - 1, 6).astype(int)])


@pytest.mark.parametrize("act", [fq.SILU, fq.GELU])
@pytest.mark.parametrize("M,F,K", TILED)
def test_forward_tiled_forms(orc, M, F, K, act):
    x, g, u = quant(orc, M, K, M, 1.0), quant(orc, F, K, F + 7, 0.05), quant(orc, F, K, F + 9, 0.05)
    forward_check(orc, x, g, u, act, save=True, pad=5, rows=some_rows(M))
    forward_check(orc, x, g, u, act, save=False, rows=some_rows(M))


def test_forward_deep_and_wide(orc):
    x, g, u = quant(orc, 40, 5120, 1, 1.0), quant(orc, 384, 5120, 2, 0.02), quant(orc, 384, 5120, 3, 0.02)
    forward_check(orc, x, g, u, fq.SILU, save=True)


def test_packed_weights_and_default_outputs(orc):
    """Gate and up as the row halves of one array, F odd: the second half's
    scales start on a 2-byte boundary; save returns halves of one buffer."""
    for M, F, K in ((70, 45, 192), (5, 45, 192), (300, 77, 640)):
        x = quant(orc, M, K, 3, 1.0)
        wc, ws = quant(orc, 2 * F, K, 4, 0.05)
        wcd, wsd = dev(wc), dev(ws)
        h, gate, up = fq.gemm_gated(dev(x[0]), dev(x[1]), wcd[:F], wsd[:F], wcd[F:], wsd[F:], save=True)
        want = forward_check(orc, x, (wc[:F], ws[:F]), (wc[F:], ws[F:]), fq.SILU, save=True)
        for a, b in zip((h, gate, up), want):
            assert np.array_equal(host_bits(a), host_bits(b))
        assert gate.stride(0) == 2 * F and up.data_ptr() == gate.data_ptr() + 2 * F


def test_nan_scale_reaches_its_row_or_column_only(orc):
    M, F, K = 40, 70, 256
    x, g, u = quant(orc, M, K, 1, 1.0), quant(orc, F, K, 2, 0.05), quant(orc, F, K, 3, 0.05)
    ref = fq.gemm_gated(*(dev(t) for t in (*x, *g, *u)))
    x[1][7, 3] = 255
    u[1][11, 0] = 255
    h = fq.gemm_gated(*(dev(t) for t in (*x, *g, *u)))
    torch.cuda.synchronize()
    nan = torch.isnan(h).cpu().numpy()
    want = np.zeros((M, F), bool)
    want[7] = want[:, 11] = True
    assert np.array_equal(nan, want)
    assert np.array_equal(host_bits(h)[~want], host_bits(ref)[~want])


def grad_check(orc, M, F, K, act, pad=0, packed=True, rows=None, sd=1.0):
    y, w = quant(orc, M, K, M + 1, 1e-3), quant(orc, F, K, F + 3, 0.05)
    rng = np.random.default_rng(M * 31 + F)
    gu = orc.round_bf16(rng.normal(0, sd, (M, 2 * F)))
    if not packed:
        gate, up = dev_bf16(gu[:, :F]), dev_bf16(gu[:, F:])
    else:
        d = dev_bf16(gu)
        gate, up = d[:, :F], d[:, F:]
    t, dg = filled(M, F, F + pad)
    t2, du = filled(M, F, F + pad)
    fq.gemm_gated_grad(dev(y[0]), dev(y[1]), dev(w[0]), dev(w[1]), gate, up, act=act, d_gate=dg, d_up=du)
    torch.cuda.synchronize()
    sel = np.arange(M) if rows is None else rows
    D, S = orc.gemm_dense(*y, *w, rows=sel)
    G, U = (orc.bf16_to_f64(np.ascontiguousarray(q[sel])) for q in (gu[:, :F], gu[:, F:]))
    s, z, dz = ob.act_parts(G, act)
    wg, wu = ob.gated_grad(D, G, U, act)
    e = act_tol(z)
    slope = ob.act_slope(G, act)
    # s (1 - s): 1 - s is off by s's error and a rounding; z' and the products by a few more
    eslope = s * e + np.abs(G * dz) * s * (2 * e + 2.0 ** -22) + 8 * ob.EPS32 * np.abs(slope)
    what = f"gated grad M={M} F={F} K={K} act={act}"
    for b in (t, t2):
        assert (host_bits(b)[:, F:] == NAN16).all(), f"{what}: wrote past F"
    tol = GEMM_REL * S
    bracket(host_bits(du)[sel], wu, tol * np.abs(G * s) + np.abs(D * G * s) * (e + 4 * ob.EPS32), orc,
            what + " d_up")
    bracket(host_bits(dg)[sel], wg, np.abs(U) * (tol * (np.abs(slope) + eslope) + np.abs(D) * eslope)
            + 4 * ob.EPS32 * np.abs(wg), orc, what + " d_gate")


@pytest.mark.parametrize("act", [fq.SILU, fq.GELU])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_grad(orc, M, F, K, act):
    grad_check(orc, M, F, K, act, pad=8, packed=False)
    grad_check(orc, M, F, K, act, pad=1)


@pytest.mark.parametrize("act", [fq.SILU, fq.GELU])
@pytest.mark.parametrize("M,F,K", [(1100, 2000, 448), (1100, 3900, 320), (1500, 5000, 128), (3000, 5900, 1152),
                                   (4100, 4400, 192)])
def test_grad_tiled_forms(orc, M, F, K, act):
    grad_check(orc, M, F, K, act, pad=3, rows=some_rows(M))


@pytest.mark.parametrize("M,F,K", [(40, 300, 2112), (200, 100, 1088), (70, 200, 4160), (500, 70, 320),
                                   (3, 6000, 192), (2500, 5, 128), (700, 7, 64)])
def test_small_tiles_and_short_rows(orc, M, F, K):
    """Each tile of the small form, and rows of fewer than 8 elements."""
    x, g, u = quant(orc, M, K, M, 1.0), quant(orc, F, K, F + 7, 0.05), quant(orc, F, K, F + 9, 0.05)
    for act in (fq.SILU, fq.GELU):
        forward_check(orc, x, g, u, act, save=True, pad=1, rows=some_rows(M))
        grad_check(orc, M, F, K, act, pad=1, rows=some_rows(M))


@pytest.mark.parametrize("act", [fq.SILU, fq.GELU])
def test_grad_far_arguments(orc, act):
    """Gates far out on both sides: the sigmoid's ends and products that vanish."""
    grad_check(orc, 33, 100, 128, act, sd=12.0)


def test_grad_block_size(orc):
    grad_check(orc, 1100, 1408, 2048, fq.SILU, rows=np.array([0, 1, 255, 256, 700, 1099]))


def test_grad_matches_differences_of_the_forward_formula(orc):
    """The gradient of sum(D * act(G) U) by central differences in float64 at
    the kernel's own (bf16) G and U."""
    M, F, K = 4, 6, 64
    y, w = quant(orc, M, K, 2, 1.0), quant(orc, F, K, 3, 0.5)
    D, S = orc.gemm(*y, *w)
    rng = np.random.default_rng(0)
    g, u = (orc.round_bf16(rng.normal(0, 1, (M, F))) for _ in range(2))
    for act in (fq.SILU, fq.GELU):
        dg, du = fq.gemm_gated_grad(dev(y[0]), dev(y[1]), dev(w[0]), dev(w[1]), dev_bf16(g), dev_bf16(u),
                                    act=act)
        torch.cuda.synchronize()
        G, U = orc.bf16_to_f64(g), orc.bf16_to_f64(u)
        e = 1e-5
        fg = (ob.gated(G + e, U, act) - ob.gated(G - e, U, act)) / (2 * e) * D
        fu = (ob.gated(G, U + e, act) - ob.gated(G, U - e, act)) / (2 * e) * D
        # half a bf16 step, the product's bound, the differences' own error (e^2 |f'''|, below 4)
        for got, want, scale in ((dg, fg, np.abs(U) * 1.2), (du, fu, np.abs(ob.act_value(G, act)))):
            v = orc.bf16_to_f64(host_bits(got))
            assert (np.abs(v - want) <= 2.0 ** -8 * np.abs(want) + GEMM_REL * S * scale
                    + np.abs(D) * (1 + np.abs(U)) * 1e-8).all()


def test_other_stream_and_graph_replays(orc):
    """Both calls on a side stream, and captured: every replay, with eager
    work between, equals the eager result."""
    M, F, K = 200, 300, 256
    x, g, u = quant(orc, M, K, 1, 1.0), quant(orc, F, K, 2, 0.05), quant(orc, F, K, 3, 0.05)
    ops = [dev(t) for t in (*x, *g, *u)]
    y, w = [dev(t) for t in quant(orc, M, K, 4, 1e-3)], [dev(t) for t in quant(orc, F, K, 5, 0.05)]

    def step(stream=None):
        h, gate, up = fq.gemm_gated(*ops, save=True, stream=stream)
        return (h, gate, up, *fq.gemm_gated_grad(*y, *w, gate, up, stream=stream))
    want = [host_bits(t) for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(np.array_equal(host_bits(a), b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host_bits(a), b) for a, b in zip(out, want))
        step()
