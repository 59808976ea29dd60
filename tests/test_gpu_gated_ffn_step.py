"""The example's training step, whole: its gradients against the same block
in float64 on the same quantised operands' values, and a fit that learns."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(HERE), "examples", "gated_ffn_step.py")
    spec = importlib.util.spec_from_file_location("gated_ffn_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def values(q):
    return fq.dequantize(*q, out_dtype=torch.float32).double().cpu().numpy()


def test_step_matches_the_block_in_float64(ex):
    """Each stage from the stage's own inputs: a product is off by at most 1e-5
    of its absolute sum and a bf16 result by half a step (2^-8) more."""
    M, H, F = 128, 64, 192
    block = ex.GatedFFN(H, F, seed=5)
    x = torch.randn(M, H, device="cuda").bfloat16()
    y, kept = block.forward(x)
    _, rstd, nT, hT, gate, up = kept
    gu = values(block.gu)
    half = 2.0 ** -8
    nq = values(fq.quantize(fq.layer_norm(x, block.copies[2], kind=fq.RMS_NORM)[0]))
    for got, w in ((gate, gu[:F]), (up, gu[F:])):
        want, S = nq @ w.T, np.abs(nq) @ np.abs(w).T
        assert (np.abs(got.double().cpu().numpy() - want) <= 1e-5 * S * (1 + half) + half * np.abs(want)).all()
    dy = (torch.randn(M, H, device="cuda") * 1e-2).bfloat16()
    dx = block.backward(dy, kept)
    torch.cuda.synchronize()
    # the weight gradient of the down projection, from the stochastic codes
    dT = fq.quantize(dy, axis=fq.COL, rounding=fq.SR, seed=1)
    a, b = values(dT), values(hT)
    assert (np.abs(block.grads[1].double().cpu().numpy() - a @ b.T) <= 1e-5 * (np.abs(a) @ np.abs(b).T)).all()
    assert dx.shape == x.shape and torch.isfinite(dx).all()
    assert all(torch.isfinite(g).all() and g.abs().max() > 0 for g in block.grads)
    # the update follows the formula from the gradients just made
    before = [p.double().cpu().numpy() for p in block.params]
    block.update(1e-2)
    for p, g, q, wd in zip(before, block.grads, block.params, (0.01, 0.01, 0.0)):
        want = ob.adamw(p, g.double().cpu().numpy(), 0.0, 0.0, 1e-2, 0.9, 0.95, 1e-8, 1, wd)[0]
        # first step: the update is lr g / (|g| + eps), off by a few roundings of fp32
        assert (np.abs(q.double().cpu().numpy() - want) <= 2.0 ** -24 * 4 * np.abs(p) + 1e-2 * 2.0 ** -19).all()
    assert all(torch.equal(c, p.bfloat16()) for c, p in zip(block.copies, block.params))


def test_fp4_gradients_point_along_the_exact_ones(ex):
    """Direction against autograd of the unquantised block in float64: an FP4
    operand is off by at most 1/8 of itself on average over a block, so the
    products of a few such keep well above half of the direction."""
    M, H, F = 512, 256, 704
    block = ex.GatedFFN(H, F, seed=7)
    x = torch.randn(M, H, device="cuda").bfloat16()
    _, kept = block.forward(x)
    dy = (torch.randn(M, H, device="cuda") * 1e-2).bfloat16()
    dx = block.backward(dy, kept)
    P = [p.double().cpu().requires_grad_() for p in block.params]
    X = x.double().cpu().requires_grad_()
    n = X * torch.rsqrt((X * X).mean(1, keepdim=True) + 1e-5) * P[2]
    z = n @ P[0].T
    y = X + (torch.nn.functional.silu(z[:, :F]) * z[:, F:]) @ P[1].T
    y.backward(dy.double().cpu())
    for got, want in zip((*block.grads, dx), (*(p.grad for p in P), X.grad)):
        cos = torch.nn.functional.cosine_similarity(got.double().cpu().flatten(), want.flatten(), dim=0)
        assert cos > 0.8, cos


@pytest.mark.parametrize("bits", [8, 32])
def test_fit_learns(ex, bits):
    losses = ex.fit(tokens=512, width=256, hidden=704, steps=40, lr=2e-3, bits=bits, report=lambda _: None)
    assert np.isfinite(losses).all()
    assert np.mean(losses[-5:]) < 0.75 * np.mean(losses[:5])
