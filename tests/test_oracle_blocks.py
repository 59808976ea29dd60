"""Pins of the block oracle (gated feed-forward, norms, AdamW): against finite
differences, double-precision autograd, published known answers and format
tables, none of them the oracle's own formulas."""
import numpy as np
import pytest
import torch

from oracle import blocks as ob


@pytest.mark.parametrize("act", [ob.SILU, ob.GELU])
def test_activation_matches_torch_in_double(act):
    g = np.linspace(-30, 30, 4001)
    t = torch.tensor(g, requires_grad=True)
    f = torch.nn.functional
    want = f.silu(t) if act == ob.SILU else f.gelu(t, approximate="tanh")
    want.sum().backward()
    assert np.allclose(ob.act_value(g, act), want.detach().numpy(), rtol=1e-11, atol=1e-13)
    assert np.allclose(ob.act_slope(g, act), t.grad.numpy(), rtol=1e-9, atol=1e-12)


@pytest.mark.parametrize("act", [ob.SILU, ob.GELU])
def test_gated_grad_matches_differences(act):
    rng = np.random.default_rng(act)
    G, U, D = rng.normal(size=(3, 5, 7))
    dG, dU = ob.gated_grad(D, G, U, act)
    h = 1e-6
    for i, j in ((0, 0), (2, 3), (4, 6)):
        e = np.zeros_like(G)
        e[i, j] = h
        fg = ((ob.gated(G + e, U, act) - ob.gated(G - e, U, act)) * D).sum() / (2 * h)
        fu = ((ob.gated(G, U + e, act) - ob.gated(G, U - e, act)) * D).sum() / (2 * h)
        assert abs(fg - dG[i, j]) < 1e-8 and abs(fu - dU[i, j]) < 1e-8


@pytest.mark.parametrize("rms", [False, True])
def test_norm_matches_double_autograd_and_differences(rms):
    rng = np.random.default_rng(7)
    x, dy = rng.normal(size=(2, 6, 33))
    x = x * 3 + 1
    w, b = rng.normal(size=(2, 33))
    eps = 1e-5
    y, mean, rstd = ob.norm(x, w, b, eps, rms)
    dx, dw, db = ob.norm_grad(dy, x, w, mean, rstd, rms)
    X, W, B = (torch.tensor(t, requires_grad=True) for t in (x, w, b))
    if rms:
        Y = X / torch.sqrt((X * X).mean(1, keepdim=True) + eps) * W + B
    else:
        Y = torch.nn.functional.layer_norm(X, (33,), W, B, eps)
    Y.backward(torch.tensor(dy))
    assert np.allclose(y, Y.detach().numpy(), rtol=0, atol=1e-12)
    for got, want in ((dx, X.grad), (dw, W.grad), (db, B.grad)):
        assert np.allclose(got, want.numpy(), rtol=0, atol=1e-12)
    h = 1e-6
    e = np.zeros_like(x)
    e[3, 5] = h
    diff = ((ob.norm(x + e, w, b, eps, rms)[0] - ob.norm(x - e, w, b, eps, rms)[0]) * dy).sum()
    assert abs(diff / (2 * h) - dx[3, 5]) < 1e-7


def test_e4m3_table_matches_the_format():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ob.e4m3_table(), want, equal_nan=True)
    assert np.nanmax(ob.e4m3_table()) == 448.0


def test_scale_byte_puts_the_largest_in_the_top_binade():
    rng = np.random.default_rng(0)
    a = np.concatenate([2.0 ** rng.uniform(-100, 100, 4000), 2.0 ** np.arange(-110.0, 100.0),
                        np.nextafter(2.0 ** np.arange(-110.0, 100.0), 0)])
    y = a / 2.0 ** (ob.e4m3_scale_byte(a) - 127.0)
    assert (y >= 128).all() and (y < 256).all()
    assert ob.e4m3_scale_byte(0.0) == 0 and ob.e4m3_scale_byte(2.0 ** -140) == 0


def test_stochastic_rounding_is_unbiased_and_stays_between_neighbours():
    u = np.arange(65536)
    for y in (0.0, 2.0 ** -9, 0.0007, 0.0031, 0.0156, 0.3, 1.06, 17.3, 255.9, 256.0):
        v = ob.e4m3_table()[ob.sr_e4m3(np.full(65536, y), u)]
        step = 2.0 ** (max(np.floor(np.log2(y)) if y else -9, -6) - 3)
        assert abs(v.mean() - y) <= step * 2.0 ** -16 + 1e-15
        assert np.abs(v - y).max() < step and len(np.unique(v)) <= 2


def test_philox_words_match_the_known_answer_generator(orc):
    seed = 0x0123456789ABCDEF
    pos = np.array([0, 1, 2, 3, 4, 1023, (1 << 34) + 7, (1 << 40) - 1], np.uint64)
    got = ob.philox_words(pos, 77, seed)
    for p, w in zip(pos.tolist(), got.tolist()):
        n = p >> 2
        want = orc.philox4x32([n & 0xFFFFFFFF, n >> 32, 77, 0], [seed & 0xFFFFFFFF, seed >> 32])
        assert w == want[p & 3]


def test_adamw_matches_torch_in_double():
    rng = np.random.default_rng(3)
    p0 = rng.normal(size=50)
    P = torch.nn.Parameter(torch.tensor(p0))
    opt = torch.optim.AdamW([P], lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.normal(size=50)
        P.grad = torch.tensor(g)
        opt.step()
        p, m, v, _, _ = ob.adamw(p, g, m, v, 1e-2, 0.9, 0.95, 1e-8, t, 0.1)
        assert np.allclose(p, P.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_nearest_rounding_stalls_an_average_and_stochastic_does_not():
    """Why the 8-bit states round stochastically: an average with beta 0.99
    pulled from 208 towards 190 stays at 208 under nearest rounding."""
    table = ob.e4m3_table()[:127]
    beta, target = 0.99, 190.0
    near, s = 208.0, np.full(4000, 208.0)
    rng = np.random.default_rng(0)
    for _ in range(600):
        near = table[np.abs(table - (beta * near + (1 - beta) * target)).argmin()]
        s = table[ob.sr_e4m3(beta * s + (1 - beta) * target, rng.integers(0, 65536, 4000))]
    assert near == 208.0
    # 0.99^600 of the start is left; the mean's noise is below 16 / sqrt(4000)
    assert abs(s.mean() - target) < 18 * 0.99 ** 600 + 5 * 16 / np.sqrt(4000)
