"""The residual norms where their launches, workgroups and teams of waves divide
the work: rows longer than one launch joins, gates whose rows do not go round,
results on their operands' memory."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq

pytestmark = pytest.mark.gpu


def test_column_sums_of_rows_beyond_one_launch():
    """2^27 columns and more are joined by more than one launch.  One row, both
    rstd 1: dbias is dy, dweight the product of two bf16, dpost_bias D, which dx
    rounds, dpost_weight its product with the branch; all exact."""
    C = (1 << 28) + 40
    dy, dxo, x, b = (torch.randn(1, C, device="cuda").bfloat16() for _ in range(4))
    one = torch.ones(1, device="cuda")
    dx, _, dw, dc, dpw, dpc, _ = fq.residual_norm_grad(
        dy, dxo, x, b, (None, one, None, one), kind=fq.RMS_NORM, post_kind=fq.RMS_NORM, want_post_weight=True,
        want_post_bias=True)
    torch.cuda.synchronize()
    assert torch.equal(dc, dy[0].float()) and torch.equal(dw, dy[0].float() * x[0].float())
    assert torch.equal(dx[0], dpc.bfloat16()) and torch.equal(dpw, dpc * b[0].float())
    assert torch.isfinite(dpc).all() and dpc[-40:].any()
