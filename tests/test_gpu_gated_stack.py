"""The residual norms, the gradient norm and the calls around them in the
stack's training step: every join from its own inputs in float64, the
gradients' direction against autograd of the unquantised stack, the clipped
update, and the step captured into a graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob
from gpu_helpers import host_bits

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
HALF = 2.0 ** -8   # half a step of bf16
# fp32 sums of 64 to 256 terms and a few roundings, 2^-24 each, twice: below this
F32 = 600 * 2.0 ** -24


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(HERE), "examples", "gated_stack.py")
    spec = importlib.util.spec_from_file_location("gated_stack", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.double().cpu().numpy()


def grads_like(x, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(x.shape, generator=g, device="cuda") * 1e-2).bfloat16()


def test_forward_joins_match_float64(ex):
    s = ex.GatedStack(64, 192, 3, seed=5)
    x = torch.randn(128, 64, device="cuda").bfloat16()
    n, kept = s.forward(x)
    for i in range(3):
        before, (after, b, stats, *_) = kept[i][0], kept[i + 1]
        _, _, post, gate, w = (f64(c) for c in s.copies[1 + 5 * i:6 + 5 * i])
        xv, bv = f64(before), f64(b)
        wx, wy, (_, pr, _, r) = ob.residual_norm(xv, bv, 1, post, None, gate[None], 128, 1.0, 1.0, True, w, None, 1e-5)
        mag = np.abs(xv) + np.abs(wx - xv)
        assert (np.abs(f64(after) - wx) <= HALF * np.abs(wx) + 2 * F32 * mag).all()
        assert np.allclose(f64(stats[1]), pr, rtol=F32, atol=0) and np.allclose(f64(stats[3]), r, rtol=2 * F32, atol=0)
    assert (np.abs(f64(n) - wy) <= HALF * np.abs(wy) + 4 * F32 * mag * r[:, None] * np.abs(w)).all()
    # without a gradient: the same up to codes that fall on the other side of a tie
    got = s.infer(x)
    assert got.shape == n.shape and got.dtype == n.dtype
    cos = torch.nn.functional.cosine_similarity(got.float().flatten(), n.float().flatten(), dim=0)
    assert cos > 0.98
    assert torch.equal(x, kept[0][0])


def test_gradients_point_along_the_exact_ones(ex):
    """Direction against autograd of the unquantised stack in float64: an FP4
    operand is off by at most 1/8 of itself on average over a block, so the
    products of a few such keep well above half of the direction."""
    M, H, F, depth = 512, 128, 320, 2
    s = ex.GatedStack(H, F, depth, seed=7)
    x = torch.randn(M, H, device="cuda").bfloat16()
    n, kept = s.forward(x)
    dn = grads_like(n)
    dx = s.backward(dn, kept)
    P = [p.double().cpu().requires_grad_() for p in s.params]
    X = x.double().cpu().requires_grad_()

    def rms(t, w):
        return t * torch.rsqrt((t * t).mean(1, keepdim=True) + 1e-5) * w
    stream, y = X, rms(X, P[0])
    for i in range(depth):
        gu, d, post, gate, w = P[1 + 5 * i:6 + 5 * i]
        z = y @ gu.T
        b = (torch.nn.functional.silu(z[:, :F]) * z[:, F:]) @ d.T
        stream = stream + gate * rms(b, post)
        y = rms(stream, w)
    y.backward(dn.double().cpu())
    for k, (got, want) in enumerate(zip((*s.grads, dx), (*(p.grad for p in P), X.grad))):
        cos = torch.nn.functional.cosine_similarity(got.double().cpu().flatten(), want.flatten(), dim=0)
        assert cos > 0.7, (k, cos)


def test_clipped_update_follows_the_formula(ex):
    s = ex.GatedStack(64, 192, 2, bits=32, seed=3)
    x = torch.randn(128, 64, device="cuda").bfloat16()
    n, kept = s.forward(x)
    s.backward(grads_like(n), kept)
    want = ob.grad_norm([f64(g) for g in s.grads], False)
    before, bound = [f64(p) for p in s.params], 0.25 * want
    norm = s.update(1e-2, bound)
    assert abs(norm.item() - want) <= 2.0 ** -23 * want
    scale = ob.clip_scale(want, bound, 1e-6)
    for p, g, q, wd in zip(before, s.grads, s.params, [0.0] + 2 * [0.01, 0.01, 0.0, 0.0, 0.0]):
        w = ob.adamw(p, f64(g), 0.0, 0.0, 1e-2, 0.9, 0.95, 1e-8, 1, wd, scale)[0]
        # the first step's update is lr g / (|g| + eps): a few roundings of fp32, and where |g| is
        # near eps the scale's half step too
        assert (np.abs(f64(q) - w) <= 2.0 ** -22 * np.abs(p) + 1e-2 * 2.0 ** -19).all()


def test_step_in_a_graph(ex):
    """Forward, backward and the norm, captured: every replay gives the eager
    step's bits, with eager work of the same calls between replays."""
    s = ex.GatedStack(64, 192, 2, seed=9)
    x = torch.randn(192, 64, device="cuda").bfloat16()
    dn = grads_like(x, 1)

    def step():
        n, kept = s.forward(x)
        dx = s.backward(dn, kept)
        return (n, dx, *s.grads, *fq.grad_norm(s.plan, 0.5))
    want = [host_bits(t.clone()) for t in step()]
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


@pytest.mark.parametrize("bits", [8, 32])
def test_runs(ex, bits):
    lines = []
    losses = ex.fit(tokens=128, width=64, hidden=192, depth=2, steps=3, bits=bits, report=lines.append)
    assert len(lines) == 3 and np.isfinite(losses).all()
