"""The norms where their kernels walk: rows longer and more numerous than one
launch, workgroup or turn of the loop takes.  Bounds as in test_gpu_norm.py."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from graph_nodes import launches
from test_gpu_norm import KINDS, TYPES, backward, forward

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


def turns(R, launch):
    """Rows that the launch's busiest walker takes: a workgroup, or each of its
    four waves where a wave holds a row (template argument MULTI = 0)."""
    walkers = launch.grid[0] * (1 if launch.args[2] else 4)
    return -(-R // walkers)


def norm_launch(R, C, xdt, ydt, kind):
    x, y = torch.empty(R, C, dtype=xdt, device="cuda"), torch.empty(R, C, dtype=ydt, device="cuda")
    one, = launches(lambda: fq.layer_norm(x, y=y, kind=kind))
    return one


def grad_launch(R, C, xdt, dydt, kind):
    x, dy = torch.empty(R, C, dtype=xdt, device="cuda"), torch.empty(R, C, dtype=dydt, device="cuda")
    s = torch.empty(R, device="cuda")
    first, *join = launches(lambda: fq.layer_norm_grad(dy, x, None, s, s, kind=kind))
    assert [j.kernel for j in join] == ["norm_grad_join_kernel"]
    return first


# MULTI, NV: a row to a wave or to a workgroup, one chunk per lane or two
WALKS = [((0, 1), 14000, 96), ((0, 1), 25001, 500), ((0, 2), 13001, 700), ((1, 1), 5001, 1111), ((1, 1), 6200, 1030),
         ((1, 1), 1301, 5120), ((1, 1), 900, 8191), ((1, 2), 601, 13824), ((1, 2), 1200, 8200)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form,R,C", WALKS)
def test_forward_walkers_take_several_rows(form, R, C, kind):
    """Rows fetched ahead, sums that alternate between two sets, statistics
    stored a row late: at least three rows to a walker."""
    for xdt, ydt in TYPES[:2] if R * C > 4e6 else TYPES:
        one = norm_launch(R, C, xdt, ydt, kind)
        assert one.kernel == "norm_kernel" and one.args[2:] == form and turns(R, one) >= 3
        forward(R, C, xdt, ydt, kind)


GRAD_WALKS = [((0, 1), 7000, 96, 4), ((0, 1), 13001, 72, 8), ((0, 1), 40000, 24, 8), ((0, 2), 1100, 1000, 4),
              ((0, 2), 2003, 800, 4), ((0, 2), 13001, 521, 8), ((1, 1), 1998, 1111, 8), ((1, 1), 5001, 2048, 16),
              ((1, 1), 1300, 8192, 8), ((1, 1), 800, 5121, 3), ((1, 2), 601, 9000, 3), ((1, 2), 700, 13824, 3),
              ((1, 2), 1100, 8200, 8)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form,R,C,least", GRAD_WALKS)
def test_backward_walkers_take_several_rows(form, R, C, least, kind):
    for xdt, dydt in TYPES[:2] if R * C > 2e6 else TYPES:
        one = grad_launch(R, C, xdt, dydt, kind)
        assert one.kernel == "norm_grad_kernel" and one.args[2:] == form and turns(R, one) >= least
        backward(R, C, xdt, dydt, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form,R,C", [((0, 1), 7001, 90), ((0, 2), 1100, 999), ((1, 1), 1998, 1111), ((1, 1), 1300, 4099),
                                      ((1, 2), 601, 8999)])
def test_backward_walks_in_place(form, R, C, kind):
    """dx over dy, and over x: a row is fetched whole before any of it is written."""
    for xdt, dydt in ((torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                      (torch.bfloat16, torch.float32)):
        assert grad_launch(R, C, xdt, dydt, kind).args[2:] == form
        backward(R, C, xdt, dydt, kind, pad=3, inplace=True)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_outside_the_registers_walk_too(kind):
    """Rows below 8 columns, more of them than workgroups."""
    for dt in (torch.float32, torch.bfloat16):
        one = norm_launch(140001, 5, dt, dt, kind)
        assert one.kernel == "norm_any_kernel" and one.grid[0] < 140001 // 2
        forward(140001, 5, dt, dt, kind)
        backward(140001, 5, dt, dt, kind)
