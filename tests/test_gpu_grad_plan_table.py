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
