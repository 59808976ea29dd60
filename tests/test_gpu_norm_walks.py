"""The norms where their kernels walk: rows longer and more numerous than one
launch, workgroup or turn of the loop takes.  Bounds as in test_gpu_norm.py."""
import numpy as np
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq

pytestmark = pytest.mark.gpu


def test_column_sums_of_rows_beyond_one_launch():
    """2^26 columns and more are joined by more than one launch.  One row with
    rstd = 1: dbias is dy and dweight the product of two bf16, both exact."""
    C = (1 << 26) + 40
    x, dy = (torch.randn(1, C, device="cuda").bfloat16() for _ in range(2))
    one = torch.ones(1, device="cuda")
    dx, dw, db = fq.layer_norm_grad(dy, x, None, None, one, kind=fq.RMS_NORM)
    torch.cuda.synchronize()
    assert torch.equal(db, dy[0].float()) and torch.equal(dw, dy[0].float() * x[0].float())
    assert torch.isfinite(dx).all()
