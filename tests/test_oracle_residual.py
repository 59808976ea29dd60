"""Pins of the oracle's residual norms and gradient norm: double-precision
autograd and finite differences of the composition, torch's norms."""
import numpy as np
import pytest
import torch

from oracle import blocks as ob

EPS = 1e-5


def torch_norm(x, w, c, kind):
    if kind == 0:
        x = x - x.mean(1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    y = y if w is None else y * w
    return y if c is None else y + c


def case(seed, R, C, groups):
    g = np.random.default_rng(seed)
    v = {k: g.normal(size=(R, C)) for k in ("x", "b", "dy", "dxo")}
    v.update({k: g.normal(size=C) for k in ("pw", "pc", "w", "c")})
    v["gate"] = g.normal(size=(groups, C)) if groups else None
    return v


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("groups,each", [(0, 7), (1, 7), (3, 3), (7, 1)])
def test_matches_double_autograd(post, rms, groups, each):
    R, C, xs, bs = 7, 19, 0.75, 0.3
    v = case(groups + 10 * post, R, C, groups)
    if post == 2:
        v["pw"] = v["pc"] = None
    t = {k: None if a is None else torch.tensor(a, requires_grad=True) for k, a in v.items()}
    n = t["b"] if post == 2 else torch_norm(t["b"], t["pw"], t["pc"], post)
    if groups:
        n = n * t["gate"][torch.arange(R) // each]
    xo = xs * t["x"] + bs * n
    y = torch_norm(xo, t["w"], t["c"], int(rms))
    ((y * t["dy"]).sum() + (xo * t["dxo"]).sum()).backward()
    gx, gy, stats = ob.residual_norm(v["x"], v["b"], post, v["pw"], v["pc"], v["gate"], each, xs, bs, rms, v["w"],
                                     v["c"], EPS)
    assert np.allclose(gx, xo.detach(), rtol=0, atol=1e-12) and np.allclose(gy, y.detach(), rtol=0, atol=1e-11)
    got = ob.residual_norm_grad(v["dy"], v["dxo"], gx, v["b"], stats, post, v["pw"], v["pc"], v["gate"], each, xs,
                                bs, rms, v["w"])
    names = dict(dx="x", dbranch="b", dweight="w", dbias="c", dpost_weight="pw", dpost_bias="pc", dgate="gate")
    assert set(got) == {k for k, n in names.items() if t[n] is not None}
    for k, a in got.items():
        assert np.allclose(a, t[names[k]].grad, rtol=0, atol=1e-10), k
    # no gradient along the stream
    alone = ob.residual_norm_grad(v["dy"], None, gx, v["b"], stats, post, v["pw"], v["pc"], v["gate"], each, xs, bs,
                                  rms, v["w"])
    assert np.allclose(got["dx"] - alone["dx"], xs * v["dxo"], atol=1e-12)


def test_matches_differences():
    R, C, each = 5, 11, 2
    v = case(3, R, C, 3)

    def loss(**kw):
        u = {**v, **kw}
        xo, y, _ = ob.residual_norm(u["x"], u["b"], 0, u["pw"], u["pc"], u["gate"], each, 0.9, 0.4, False, u["w"],
                                    u["c"], EPS)
        return (y * v["dy"]).sum() + (xo * v["dxo"]).sum()
    xo, _, stats = ob.residual_norm(v["x"], v["b"], 0, v["pw"], v["pc"], v["gate"], each, 0.9, 0.4, False, v["w"],
                                    v["c"], EPS)
    got = ob.residual_norm_grad(v["dy"], v["dxo"], xo, v["b"], stats, 0, v["pw"], v["pc"], v["gate"], each, 0.9,
                                0.4, False, v["w"])
    for k, name in (("dx", "x"), ("dbranch", "b"), ("dgate", "gate"), ("dpost_weight", "pw"), ("dpost_bias", "pc")):
        for i in range(0, v[name].size, 7):
            e = np.zeros(v[name].size)
            e[i] = 1e-6
            e = e.reshape(v[name].shape)
            d = (loss(**{name: v[name] + e}) - loss(**{name: v[name] - e})) / 2e-6
            assert abs(d - got[k].ravel()[i]) < 1e-6 * (1 + abs(d)), (k, i)


def test_grad_norm_matches_torch():
    g = [torch.randn(n, dtype=torch.float64) for n in (1, 0, 7, 100)]
    flat = torch.cat(g)
    a = [t.numpy() for t in g]
    assert np.isclose(ob.grad_norm(a, False), torch.linalg.vector_norm(flat).item(), rtol=1e-14)
    assert ob.grad_norm(a, True) == flat.abs().max().item() and ob.grad_norm([], False) == 0.0
    p = [torch.nn.Parameter(t.clone()) for t in g]
    for q, t in zip(p, g):
        q.grad = t.clone()
    norm = torch.nn.utils.clip_grad_norm_(p, 1.5)
    scale = ob.clip_scale(norm.item(), 1.5, 1e-6)
    assert np.allclose(p[3].grad.numpy(), a[3] * scale, rtol=1e-12)
    assert ob.clip_scale(0.5, 1.5, 1e-6) == 1.0 and ob.clip_scale(0.0, 0.0, 0.0) == 1.0
    assert ob.clip_scale(np.inf, 1.0, 1e-6) == 0.0 and np.isnan(ob.clip_scale(np.nan, 1.0, 1e-6))
