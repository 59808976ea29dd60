"""The residual norms where their launches, workgroups and teams of waves divide
the work: rows longer than one launch joins, gates whose rows do not go round,
results on their operands' memory."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from test_gpu_residual_norm import BF, F32, LAYER, NONE, RMS, Case

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


@pytest.mark.parametrize("C", [300, 520, 1030, 2050])
@pytest.mark.parametrize("gates", [5, 7, 12, 13, 17, 23])
def test_gates_that_do_not_go_round(gates, C):
    """Groups that are fewer than the teams of a workgroup, or do not divide
    among them: as slabs of their own and as whole ones."""
    Case(6000 if C < 2000 else 3000, C, BF, BF, LAYER, RMS, gates=gates, gdt=F32).check_backward(BF)


def same(a, b):
    return [i for i, (x, y) in enumerate(zip(a, b)) if y is not None and not torch.equal(x, y)] == []


SHARED = [513, 519, 1025, 1543, 5121, 6139, 8185, 8200, 9217, 13825]  # two waves hold the last elements


@pytest.mark.parametrize("C", SHARED)
def test_repeated_calls_give_the_same_bits(C):
    """Elements that two waves hold, at other places of their lanes, are stored by
    both: the same bits whichever is the last, in every form of the gates."""
    R = 2600 if C < 1000 else 700
    for post, kind, gates, dt, gdt in ((RMS, LAYER, 5, BF, BF), (LAYER, RMS, 5, F32, BF), (LAYER, LAYER, 1, BF, F32),
                                       (NONE, RMS, 3, F32, F32), (LAYER, LAYER, 0, BF, BF), (RMS, RMS, R, F32, BF)):
        c = Case(R, C, dt, dt, post, kind, gates=gates, gdt=gdt, xs=0.75, bs=0.3)
        xo, y, stats = c.forward()
        dy, dxo = (torch.randn(R, C, device="cuda").to(dt) for _ in range(2))

        def back():
            return fq.residual_norm_grad(dy, dxo, xo, c.b, stats, c.w, **c.kw)
        want = back()
        for _ in range(4):
            assert same(back(), want), (C, post, kind, gates, dt)
            again = c.forward()
            assert same((*again[:2], *again[2]), (xo, y, *stats)), (C, post, kind, gates, dt)


@pytest.mark.parametrize("C", SHARED)
def test_forward_on_its_own_operand(C):
    """x_out on x's memory: the same bits as in memory of its own, with rows
    enough that every workgroup walks."""
    for post, gates, xdt, bdt in ((LAYER, 0, BF, BF), (NONE, 0, F32, F32), (NONE, 0, BF, F32), (RMS, 3, F32, BF)):
        c = Case(2600 if C < 1000 else 700, C, xdt, bdt, post, RMS if gates else LAYER, gates=gates)
        xo, y, stats = c.forward()
        for _ in range(2):
            into, c.x = c.x, c.x.clone()
            x2, y2, stats2 = fq.residual_norm(into, c.b, c.w, c.c, eps=c.eps, x_out=into, **c.kw)
            assert x2 is into and same((x2, y2, *stats2), (xo, y, *stats))


@pytest.mark.parametrize("C", SHARED)
def test_backward_on_its_own_operands(C):
    """dx on dx_out's or dy's memory and dbranch on branch's or dy's: the same
    bits as in memory of their own."""
    R = 2600 if C < 1000 else 700
    for post, gates, dt in ((LAYER, 0, BF), (NONE, 0, F32), (RMS, 5, BF)):
        c = Case(R, C, dt, dt, post, RMS if gates else LAYER, gates=gates)
        xo, _, stats = c.forward()
        dy, dxo = (torch.randn(R, C, device="cuda").to(dt) for _ in range(2))

        def run(dx, dbranch):
            """Operands by name; results on the named ones."""
            t = dict(dy=dy.clone(), dx_out=dxo.clone(), branch=c.b.clone())
            at = {k: t.get(v) for k, v in (("dx", dx), ("dbranch", dbranch))}
            out = fq.residual_norm_grad(t["dy"], t["dx_out"], xo, t["branch"], stats, c.w, **at, **c.kw)
            assert all(v is None or out[i] is v for i, v in enumerate(at.values()))
            return out
        want = run(None, None)
        for dx, dbranch in (("dx_out", "branch"), ("dy", "branch"), ("dx_out", "dy"), ("dy", None), (None, "dy")):
            assert same(run(dx, dbranch), want), (dx, dbranch)
