"""The norm of many gradients and their clipping, against float64.

The squares and sums are in 64 bits, so that the norm is the exact one rounded
to fp32: within half a step (2^-24 of it), and a hair for the sum's roundings
of 2^-53 each.  The scale is formed from the unrounded norm: half a step too."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from oracle import blocks as ob
from gpu_helpers import host_bits

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -24 * (1 + 2.0 ** -20)


def make(sizes, seed=0, sd=1e-3, dtypes=(F32, BF), packed=True):
    """Gradients behind each other in one buffer of each type (packed: at any
    element), and their float64 values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        buf = (torch.randn(n + 9, generator=g, device="cuda") * sd).to(dt)
        out.append(buf[i % 8:][:n] if packed else buf[:n].clone())
    return out


def f64(t):
    return t.double().cpu().numpy()


def check(grads, max_norm, order, eps=1e-6):
    want = ob.grad_norm([f64(t) for t in grads], order == fq.NORM_MAX)
    norm, scale = fq.grad_norm(fq.grad_plan(grads), max_norm, eps, order)
    assert norm.shape == scale.shape == ()
    assert abs(norm.item() - want) <= HALF * want
    ws = ob.clip_scale(want, max_norm, eps)
    assert abs(scale.item() - ws) <= HALF * ws
    return norm, scale


ORDERS = [fq.NORM_L2, fq.NORM_MAX]
SIZES = [[1], [0, 1, 0], [3], [7, 8, 9], [255, 256, 257], [1023, 1025, 4096], [4097, 16383], [16384, 16385, 1],
         [100000, 12345, 1], [1 << 20, 3, 65536 + 5], [3] * 191, [5] * 192, [2] * 193, [777] * 500,
         [1] * 150 + [40000] * 150]


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_scale(sizes, order):
    for dtypes in ((F32, BF), (F32,), (BF,)):
        g = make(sizes, len(sizes), dtypes=dtypes)
        n = max(ob.grad_norm([f64(t) for t in g], order == fq.NORM_MAX), 1e-6)
        for max_norm in (0.3 * n, 1.0001 * n + 1e-6, 0.0):
            check(g, max_norm, order)


def test_largest_at_either_end_and_signs():
    for n in (1, 64, 5000, 40000):
        for i in (0, n - 1, n // 2):
            for dt in (F32, BF):
                g = torch.zeros(n, device="cuda", dtype=dt)
                g[i] = -3.0
                for order in ORDERS:
                    assert fq.grad_norm(fq.grad_plan([g]), 1.0, 0.0, order)[0].item() == 3.0


@pytest.mark.parametrize("order", ORDERS)
def test_range_of_fp32(order):
    """Squares far outside fp32's range, and gradients that are not normal."""
    for v in (3e38, 1e25, 1e-25, 1e-38, 1e-44):
        g = torch.full((3000,), v, device="cuda")
        if order == fq.NORM_L2 and v == 3e38:
            g = g[:1]
        want = ob.grad_norm([f64(g)], order == fq.NORM_MAX)
        norm, scale = fq.grad_norm(fq.grad_plan([g]), 0.5 * v, 0.0, order)
        assert abs(norm.item() - want) <= HALF * want + 2.0 ** -150
        assert abs(scale.item() - 0.5 * v / want) <= HALF
    # a norm above fp32's largest is Inf, its scale still the right one
    g = torch.full((100,), 3e38, device="cuda")
    norm, scale = fq.grad_norm(fq.grad_plan([g]), 1e38, 0.0, fq.NORM_L2)
    assert norm.isinf() and abs(scale.item() - 1e38 / (10 * 3e38)) < 1e-6


@pytest.mark.parametrize("order", ORDERS)
def test_non_finite_and_empty(order):
    inf, nan = float("inf"), float("nan")
    for dt in (F32, BF):
        for values, norm, scale in (([inf], inf, 0.0), ([-inf], inf, 0.0), ([nan], nan, nan), ([inf, nan], nan, nan)):
            g = make([5000, 300], 1, dtypes=(dt,))
            for i, v in enumerate(values):
                g[i][299 - 17 * i] = v
            a, b = fq.grad_norm(fq.grad_plan(g), 1.0, order=order)
            assert np.array_equal([a.item(), b.item()], [norm, scale], equal_nan=True)
    for g in ([torch.zeros(0, device="cuda")], [torch.zeros(70, device="cuda")]):
        a, b = fq.grad_norm(fq.grad_plan(g), 1.0, order=order)
        assert (a.item(), b.item()) == (0.0, 1.0)
        a, b = fq.grad_norm(fq.grad_plan(g), 0.0, eps=0.0, order=order)
        assert (a.item(), b.item()) == (0.0, 1.0)
    a, b = fq.grad_norm(fq.grad_plan(make([10])), order=order)
    assert a.item() > 0 and b is None


@pytest.mark.parametrize("sizes", [[1], [7, 9, 8], [16385, 3, 40000], [1 << 20, 5], [11] * 400], ids=len)
def test_clipping(sizes):
    """Each element times the scale, rounded once; memory around them stays."""
    for dtypes in ((F32, BF), (BF,)):
        g = make(sizes, 3, dtypes=dtypes)
        bases = [t._base if t._base is not None else t for t in g]
        before = [b.clone() for b in bases]
        plan = fq.grad_plan(g)
        old = [t.clone() for t in g]
        n = ob.grad_norm([f64(t) for t in g], False)
        norm, scale = fq.grad_norm(plan, 0.37 * n)
        got = fq.clip_grads(plan, 0.37 * n)
        assert torch.equal(got, norm) and 0.3 < scale.item() < 0.4
        for t, o in zip(g, old):
            assert torch.equal(t, (o.float() * scale).to(t.dtype))
        for b, was, t in zip(bases, before, g):
            i = t.storage_offset()
            b[i:i + t.numel()] = was[i:i + t.numel()]
            assert torch.equal(b, was)
        # gradients within the bound stay as they are, bit for bit
        assert fq.clip_grads(plan, 2 * n).item() == norm.item()
        assert all(torch.equal(t, o) for t, o in zip(g, old))


def test_clipping_non_finite():
    g = make([300], dtypes=(F32,))[0]
    g[5], g[9] = float("inf"), -float("inf")
    fq.clip_grads(fq.grad_plan([g]), 1.0)
    bad = g.isnan()  # Inf times 0; the others become 0
    assert bad.nonzero().flatten().tolist() == [5, 9] and (g[~bad] == 0).all()
    g = make([300], dtypes=(F32,))[0]
    g[5] = float("nan")
    assert fq.clip_grads(fq.grad_plan([g]), 1.0).isnan() and g.isnan().all()


@pytest.mark.parametrize("sizes", [[16385, 3, 40000] * 20, [700] * 300, [70000]], ids=len)
def test_arguments_and_table_give_the_same_bits(sizes):
    """The C calls without a table, whose descriptors are kernel arguments."""
    g = make(sizes, 8)
    plan = fq.grad_plan(g)
    norm, scale = fq.grad_norm(plan, 0.01)
    a, b = torch.zeros(2, device="cuda").split(1)
    ws = torch.empty(plan.nbytes, dtype=torch.uint8, device="cuda")
    for order in ORDERS:
        want = fq.grad_norm(plan, 0.01, order=order)
        assert fq.lib().fp4q_grad_norm(plan.array, plan.n, None, order, 0.01, 1e-6, a.data_ptr(), b.data_ptr(),
                                       ws.data_ptr(), plan.nbytes, None) == 0
        assert torch.equal(a[0], want[0]) and torch.equal(b[0], want[1])
    old = [t.clone() for t in g]
    assert fq.lib().fp4q_grad_clip(plan.array, plan.n, None, 0, 0.01, 1e-6, a.data_ptr(), ws.data_ptr(), plan.nbytes,
                                   None) == 0
    assert torch.equal(a[0], norm)
    assert all(torch.equal(t, (o.float() * scale).to(t.dtype)) for t, o in zip(g, old))
    for t, o in zip(g, old):
        t.copy_(o)
    assert fq.lib().fp4q_grad_scale(plan.array, plan.n, None, scale.data_ptr(), None) == 0
    assert all(torch.equal(t, (o.float() * scale).to(t.dtype)) for t, o in zip(g, old))


def test_with_the_adamw_step():
    """grad_norm of an AdamW plan, its scale in the step: what a step over
    gradients clipped by hand gives."""
    sizes = [4096, 130, 7]

    def fresh():
        p, g = make(sizes, 5, 1.0, (F32,), packed=False), make(sizes, 6, 1e-2, (F32,), packed=False)
        m, v = ([torch.zeros_like(t) for t in p] for _ in range(2))
        return p, g, fq.adamw_plan(p, g, m, v)
    p, g, plan = fresh()
    norm, scale = fq.grad_norm(plan, 0.1)
    want = ob.grad_norm([f64(t) for t in g], False)
    assert abs(norm.item() - want) <= HALF * want and scale.item() < 0.2
    fq.adamw_step(plan, 1e-3, 1, grad_scale=scale)
    q, h, other = fresh()
    fq.clip_grads(other, 0.1)
    fq.adamw_step(other, 1e-3, 1)
    assert all(torch.equal(a, b) for a, b in zip(p, q))
    assert not torch.equal(g[0], h[0])


def test_large_tensor_offsets():
    """A tensor beyond 2^31 elements: the last one is found and scaled."""
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-1], g[5] = 4.0, -3.0
    plan = fq.grad_plan([g])
    assert fq.grad_norm(plan, 1.0)[0].item() == 5.0
    assert fq.grad_norm(plan, 1.0, order=fq.NORM_MAX)[0].item() == 4.0
    fq.clip_grads(plan, 2.5, eps=0.0)
    assert (g[-1].item(), g[5].item()) == (2.0, -1.5)


def test_streams_graphs_and_repeats():
    g = make([50000, 300, 16384 * 3 + 1, 7] * 60, 9)
    plan = fq.grad_plan(g)
    norm, scale = fq.grad_norm(plan, 0.1)
    for _ in range(3):
        again = fq.grad_norm(plan, 0.1)
        assert torch.equal(again[0], norm) and torch.equal(again[1], scale)
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(8):
            a @ a
    got = fq.grad_norm(plan, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], norm) and torch.equal(got[1], scale)
    old = [t.clone() for t in g]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fq.clip_grads(plan, 0.1)
    for _ in range(3):
        for t, o in zip(g, old):
            t.copy_(o)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, norm)
        assert all(torch.equal(t, (o.float() * scale).to(t.dtype)) for t, o in zip(g, old))
        fq.grad_norm(plan, 0.2)


def test_a_plan_made_inside_a_capture():
    g = make([20000, 50, 30000] * 30, 4)
    norm, scale = fq.grad_norm(fq.grad_plan(g), 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = fq.grad_plan(g)
        out = fq.grad_norm(plan, 0.1)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], norm) and torch.equal(out[1], scale)
        fq.grad_norm(plan, 0.2)


def test_refusals_on_the_device():
    plan = fq.grad_plan(make([100]))
    with pytest.raises(fq.Fp4qError, match="workspace"):
        fq.grad_norm(plan, 1.0, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fq.Fp4qError, match="max_norm"):
        fq.grad_norm(plan, -1.0)
    with pytest.raises(fq.Fp4qError, match="order"):
        fq.grad_norm(plan, 1.0, order=7)


def test_outputs_that_are_given():
    plan = fq.grad_plan(make([1000]))
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros((), device="cuda")
    a, b = fq.grad_norm(plan, 1e-3, norm=norm, scale=scale)
    want = fq.grad_norm(plan, 1e-3)
    assert a is norm and b is scale
    assert host_bits(a)[0] == host_bits(want[0]) and host_bits(b) == host_bits(want[1])
