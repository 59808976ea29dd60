"""The gated calls at sizes that take each of their kernels' forms, which the
launch itself names.  Bounds as in test_gpu_gated.py."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from graph_nodes import launches
from test_gpu_gated import forward_check, grad_check, quant, some_rows

pytestmark = pytest.mark.gpu

ACTS = [fq.SILU, fq.GELU]


def codes(rows, K):
    return [torch.empty(rows, k, dtype=torch.uint8, device="cuda") for k in (K // 2, K // 32)]


def forward_form(M, F, K, act, save):
    ops = [t for rows in (M, F, F) for t in codes(rows, K)]
    one, = launches(lambda: fq.gemm_gated(*ops, act=act, save=save))
    return one.kernel, one.args


def grad_form(M, F, K, act):
    ops = [t for rows in (M, F) for t in codes(rows, K)]
    gu = torch.empty(2, M, F, dtype=torch.bfloat16, device="cuda")
    one, = launches(lambda: fq.gemm_gated_grad(*ops, *gu, act=act))
    return one.kernel, one.args


# small tiles as (16-row, 16-column fragments, waves along K)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tile,M,F,K", [
    ((1, 1, 4), 16, 2500, 1088), ((1, 1, 4), 50, 1000, 2048), ((1, 1, 4), 100, 1030, 960),
    ((2, 1, 8), 128, 700, 2112), ((2, 1, 8), 121, 650, 1600), ((2, 1, 8), 64, 1405, 1152), ((2, 1, 8), 250, 350, 4096),
    ((2, 2, 4), 128, 1408, 960), ((2, 2, 4), 200, 1003, 1472), ((2, 2, 4), 250, 900, 512)])
def test_forward_small_tiles(orc, tile, M, F, K, act):
    x, g, u = quant(orc, M, K, M, 1.0), quant(orc, F, K, F + 7, 0.05), quant(orc, F, K, F + 9, 0.05)
    for save in (False, True):
        assert forward_form(M, F, K, act, save) == ("gated_small_kernel", (act, 0, int(save), *tile))
        forward_check(orc, x, g, u, act, save=save, pad=3, rows=some_rows(M))


# 3: 128-row tiles of four waves, 2: 256-row ones, 0: 256 x 256 of eight
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("cfg,M,F,K", [
    (3, 250, 1500, 3136), (3, 300, 1300, 4224), (3, 500, 4000, 64), (2, 1100, 1900, 3136), (2, 1100, 1900, 4160),
    (2, 1050, 2001, 2176), (0, 1100, 4000, 1600), (0, 1300, 3500, 4096)])
def test_forward_tiles(orc, cfg, M, F, K, act):
    x, g, u = quant(orc, M, K, M, 1.0), quant(orc, F, K, F + 7, 0.05), quant(orc, F, K, F + 9, 0.05)
    for save in (False, True):
        assert forward_form(M, F, K, act, save) == ("gemm_gated_kernel", (cfg, act, int(save), int(K % 128 != 0)))
        forward_check(orc, x, g, u, act, save=save, pad=0 if save else 3, rows=some_rows(M))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tile,M,F,K", [
    ((1, 2, 8), 200, 600, 3136), ((1, 2, 8), 4000, 7, 192), ((2, 2, 4), 300, 700, 320), ((2, 2, 4), 300, 700, 1024),
    ((2, 2, 4), 250, 1001, 2112), ((2, 2, 4), 5000, 7, 64), ((2, 4, 4), 512, 1408, 192), ((2, 4, 4), 3000, 200, 960),
    ((2, 4, 4), 400, 1203, 1088), ((2, 4, 4), 20000, 7, 1024), ((2, 4, 4), 20000, 1, 640)])
def test_grad_small_tiles(orc, tile, M, F, K, act):
    assert grad_form(M, F, K, act) == ("gated_small_kernel", (act, 1, 0, *tile))
    grad_check(orc, M, F, K, act, pad=3, rows=some_rows(M))
    grad_check(orc, M, F, K, act, packed=False, rows=some_rows(M))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("cfg,M,F,K", [
    (3, 1200, 1301, 2112), (3, 1230, 1400, 960), (3, 1200, 1300, 3200), (2, 1000, 5000, 3136), (2, 1000, 5001, 4160),
    (2, 1020, 4900, 2176), (0, 2000, 5003, 1600), (0, 2000, 5000, 4096)])
def test_grad_tiles(orc, cfg, M, F, K, act):
    assert grad_form(M, F, K, act) == ("gemm_gated_grad_kernel", (cfg, act, int(K % 128 != 0)))
    grad_check(orc, M, F, K, act, pad=3, rows=some_rows(M))
    grad_check(orc, M, F, K, act, rows=some_rows(M))
