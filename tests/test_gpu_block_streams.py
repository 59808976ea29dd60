"""The gated and norm calls with stream=: the same bits as on the current
stream, and results that are dropped while the stream is still busy leave
other tensors' memory alone."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from mxfp4_block_scaled_fp4q_amd import inputs
from gpu_helpers import dev, host_bits

pytestmark = pytest.mark.gpu


def busy(stream, a):
    """A few milliseconds of products on the stream."""
    with torch.cuda.stream(stream):
        for _ in range(8):
            a @ a


def quant(orc, rows, K, seed, sd):
    return [dev(t) for t in orc.quantize(inputs.normal((rows, K), seed) * np.float32(sd), 32)]


def test_stream_argument(orc):
    M, F, K = 200, 300, 256
    ops = [t for rows, seed in ((M, 1), (F, 2), (F, 3)) for t in quant(orc, rows, K, seed, 0.3)]
    back = quant(orc, M, K, 4, 1e-3) + quant(orc, F, K, 5, 0.05)
    x, dy = torch.randn(2, 1000, 520, device="cuda").bfloat16()
    w, b = torch.randn(2, 520, device="cuda")
    a = torch.randn(4096, 4096, device="cuda")

    def step(stream=None):
        h, gate, up = fq.gemm_gated(*ops, save=True, stream=stream)
        grads = fq.gemm_gated_grad(*back, gate, up, stream=stream)
        y, mean, rstd = fq.layer_norm(x, w, b, stream=stream)
        return (h, gate, up, *grads, y, mean, rstd, *fq.layer_norm_grad(dy, x, w, mean, rstd, stream=stream))
    want = [host_bits(t) for t in step()]
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        busy(side, a)
        got = step(side)
        torch.cuda.current_stream().wait_stream(side)
        for t, wanted in zip(got, want):
            assert np.array_equal(host_bits(t), wanted)


def test_dropped_results_leave_other_memory_alone():
    x = torch.randn(1000, 96, device="cuda")
    a = torch.randn(4096, 4096, device="cuda")
    want = fq.layer_norm(x)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy(side, a)
    y = fq.layer_norm(x, stream=side)[0]  # mean and rstd are dropped, unwritten as yet
    others = [torch.full((1000,), 7.0, device="cuda") for _ in range(8)]
    side.synchronize()
    assert torch.equal(y, want)
    assert all((t == 7.0).all() for t in others)
