"""Gradient plans and their tables on the device: made in and after captures,
and read by every call."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from test_gpu_grad_norm import BF, F32, make

pytestmark = pytest.mark.gpu


def test_a_plan_of_a_capture_in_eager_calls():
    """Made inside a capture, then used outside and in a second capture: the same
    bits throughout."""
    g = make([20000, 50, 30000] * 100, 4)
    norm, scale = fq.grad_norm(fq.grad_plan(g), 0.1)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        plan = fq.grad_plan(g)
        a = fq.grad_norm(plan, 0.1)
    assert plan.table is None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = fq.grad_norm(plan, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert plan.table is not None
    with torch.cuda.graph(second):
        c = fq.grad_norm(plan, 0.1)
    for _ in range(3):
        for t in (*a, *c):
            t.zero_()
        first.replay()
        second.replay()
        torch.cuda.synchronize()
        for got in (a, b, c, fq.grad_norm(plan, 0.1)):
            assert torch.equal(got[0], norm) and torch.equal(got[1], scale)


@pytest.mark.parametrize("sizes", [[1], [3, 0, 9], [700] * 300, [16385, 3, 40000] * 20, [1 << 24, 5, 1 << 20]], ids=len)
def test_scaling_by_a_device_factor(sizes):
    """scale_grads reads the plan's table: each element times the factor, rounded
    once, and memory around them as it was; 1 leaves them bit for bit."""
    for dtypes in ((F32, BF), (BF,), (F32,)):
        g = make(sizes, 12, dtypes=dtypes)
        plan = fq.grad_plan(g)
        assert plan.table is not None
        bases = [t._base if t._base is not None else t for t in g]
        before = [b.clone() for b in bases]
        for factor in (1.0, -0.37, 0.0, float("nan")):
            old = [t.clone() for t in g]
            scale = torch.tensor(factor, device="cuda")
            fq.scale_grads(plan, scale)
            for t, o in zip(g, old):
                want = o if factor == 1.0 else (o.float() * scale).to(t.dtype)
                assert torch.equal(t.isnan(), want.isnan()) and torch.equal(t.nan_to_num(7.0), want.nan_to_num(7.0))
            for b, was, t in zip(bases, before, g):
                i, n = t.storage_offset(), t.numel()
                assert torch.equal(b[:i], was[:i]) and torch.equal(b[i + n:], was[i + n:])


def test_scaling_on_another_stream_and_in_a_graph():
    g = make([50000, 300, 16384 * 3 + 1, 7] * 60, 9)
    plan, old = fq.grad_plan(g), [t.clone() for t in g]
    scale = torch.tensor(0.25, device="cuda")
    want = [(o.float() * 0.25).to(o.dtype) for o in old]
    a = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(8):
            a @ a
    fq.scale_grads(plan, scale, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(t, w) for t, w in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fq.scale_grads(plan, scale)
    for factor in (0.25, 1.0, 0.25):
        for t, o in zip(g, old):
            t.copy_(o)
        scale.fill_(factor)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w if factor < 1 else o) for t, w, o in zip(g, want, old))
        fq.grad_norm(plan, 0.1)
