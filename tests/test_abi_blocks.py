"""Refusals of the gated, norm and AdamW calls, on the host: status codes for
every bad argument, nothing launched."""
import ctypes as ct

import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq

FAKE = 0x10000   # 16-byte aligned, never dereferenced
NUL = 0


@pytest.fixture(scope="module")
def L():
    return fq.lib()


def gated(L, **kw):
    a = dict(M=64, F=48, K=128, xc=FAKE, xs=FAKE, gc=FAKE, gs=FAKE, uc=FAKE, us=FAKE, act=0, h=FAKE,
             ldh=48, gate=FAKE, up=FAKE, ld=48)
    a.update(kw)
    return L.fp4q_gemm_gated(*a.values(), NUL)


@pytest.mark.parametrize("kw,status", [
    (dict(xc=NUL), 1), (dict(us=NUL), 1), (dict(h=NUL), 1), (dict(gate=NUL), 1), (dict(up=NUL), 1),
    (dict(act=2), 1), (dict(act=-1), 1), (dict(M=0), 1), (dict(F=0), 1), (dict(F=-5), 1),
    (dict(K=0), 1), (dict(K=96), 1), (dict(M=1 << 30), 1), (dict(K=1 << 24), 2),
    (dict(M=(1 << 30) - 1, F=(1 << 30) - 1, ldh=1 << 30, ld=1 << 30), 2),
    (dict(ldh=47), 1), (dict(ld=47), 1),
    (dict(xc=FAKE + 8), 3), (dict(uc=FAKE + 8), 3), (dict(gs=FAKE + 2), 3), (dict(us=FAKE + 3), 3),
    (dict(us=FAKE + 1, K=64), 3), (dict(h=FAKE + 1), 3), (dict(up=FAKE + 1), 3),
])
def test_gemm_gated_refusals(L, kw, status):
    assert gated(L, **kw) == status
    assert "gemm_gated" in L.fp4q_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(yc=NUL), 1), (dict(gate=NUL), 1), (dict(dup=NUL), 1), (dict(act=3), 1), (dict(M=-1), 1),
    (dict(K=160), 1), (dict(K=1 << 24), 2), (dict(ld=47), 1), (dict(ldd=40), 1),
    (dict(ws=FAKE + 4), 3), (dict(yc=FAKE + 4), 3), (dict(gate=FAKE + 1), 3), (dict(dg=FAKE + 1), 3),
])
def test_gemm_gated_grad_refusals(L, kw, status):
    a = dict(M=64, F=48, K=128, yc=FAKE, ys=FAKE, wc=FAKE, ws=FAKE, act=0, gate=FAKE, up=FAKE,
             ld=48, dg=FAKE, dup=FAKE, ldd=48)
    a.update(kw)
    assert L.fp4q_gemm_gated_grad(*a.values(), NUL) == status
    assert "gemm_gated_grad" in L.fp4q_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(kind=2), 1), (dict(x=NUL), 1), (dict(y=NUL), 1), (dict(xdt=2), 1), (dict(wdt=-1), 1),
    (dict(ydt=9), 1), (dict(rows=0), 1), (dict(cols=0), 1), (dict(rows=1 << 31), 1),
    (dict(ldx=32), 1), (dict(ldy=32), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(x=FAKE + 1), 3), (dict(y=FAKE + 2, ydt=0), 3),
    (dict(w=FAKE + 2), 3), (dict(mean=FAKE + 2), 3), (dict(rstd=FAKE + 1), 3),
])
def test_layer_norm_refusals(L, kw, status):
    a = dict(kind=0, x=FAKE, xdt=1, rows=4, cols=33, ldx=33, w=FAKE, b=FAKE, wdt=0, eps=1e-5, y=FAKE,
             ydt=1, ldy=33, mean=FAKE, rstd=FAKE)
    a.update(kw)
    assert L.fp4q_layer_norm(*a.values(), NUL) == status
    assert "layer_norm" in L.fp4q_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(kind=5), 1), (dict(dy=NUL), 1), (dict(rstd=NUL), 1), (dict(mean=NUL), 1), (dict(dx=NUL), 1),
    (dict(dydt=4), 1), (dict(rows=0), 1), (dict(lddy=0), 1), (dict(ldx=32), 1), (dict(lddx=32), 1),
    (dict(ws=NUL), 1), (dict(ws=FAKE + 8), 3), (dict(nb=0), 4), (dict(dx=FAKE + 1), 3),
    (dict(dw=FAKE + 2), 3),
])
def test_layer_norm_grad_refusals(L, kw, status):
    a = dict(kind=0, dy=FAKE, dydt=1, lddy=33, x=FAKE, xdt=1, rows=4, cols=33, ldx=33, w=FAKE, wdt=0,
             mean=FAKE, rstd=FAKE, dx=FAKE, lddx=33, dw=FAKE, db=FAKE, ws=FAKE, nb=1 << 30)
    a.update(kw)
    assert L.fp4q_layer_norm_grad(*a.values(), NUL) == status
    assert "layer_norm_grad" in L.fp4q_last_error().decode()


def test_layer_norm_grad_workspace_bytes(L):
    w = L.fp4q_layer_norm_grad_workspace_bytes
    assert w(0, 5) == 0 and w(5, 0) == 0 and w(1, 1) > 0
    assert w(16384, 5120) <= 64 << 20


def tensor(**kw):
    a = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scales=FAKE,
             exp_avg_sq_scales=FAKE, copy=FAKE, numel=100, weight_decay=0.1)
    a.update(kw)
    return fq.AdamwTensor(*a.values())


def adamw(L, t, n=None, bits=32, gdt=0, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, step=1, scale=NUL):
    arr = (fq.AdamwTensor * max(len(t), 1))(*t)
    return L.fp4q_adamw_step(arr, len(t) if n is None else n, bits, gdt, lr, b1, b2, eps, step, 0,
                             scale, NUL)


@pytest.mark.parametrize("t,kw,status", [
    ({}, dict(n=-1), 1), ({}, dict(bits=16), 1), ({}, dict(gdt=2), 1), ({}, dict(lr=-1e-3), 1),
    ({}, dict(lr=float("nan")), 1), ({}, dict(b1=1.0), 1), ({}, dict(b2=1.0), 1),
    ({}, dict(b2=-0.1), 1), ({}, dict(eps=-1.0), 1), ({}, dict(step=0), 1),
    ({}, dict(step=1 << 32), 1), ({}, dict(scale=FAKE + 2), 3),
    (dict(param=NUL), {}, 1), (dict(grad=NUL), {}, 1), (dict(exp_avg_sq=NUL), {}, 1),
    (dict(exp_avg_scales=NUL), dict(bits=8), 1), (dict(numel=-1), {}, 1),
    (dict(numel=1 << 40), {}, 1), (dict(weight_decay=-0.1), {}, 1),
    (dict(weight_decay=float("nan")), {}, 1), (dict(param=FAKE + 4), {}, 3),
    (dict(grad=FAKE + 8), {}, 3), (dict(exp_avg=FAKE + 1), dict(bits=8), 3),
    (dict(copy=FAKE + 2), {}, 3),
])
def test_adamw_refusals(L, t, kw, status):
    assert adamw(L, [tensor(numel=0), tensor(**t)], **kw) == status
    assert "adamw_step" in L.fp4q_last_error().decode()


def test_adamw_null_array_and_empty_calls(L):
    assert L.fp4q_adamw_step(NUL, 3, 32, 0, 1e-3, 0.9, 0.95, 1e-8, 1, 0, NUL, NUL) == 1
    # nothing to do launches nothing
    assert adamw(L, [], n=0) == 0
    assert adamw(L, [tensor(numel=0, param=NUL)] * 100) == 0


def test_descriptor_matches_the_header():
    assert ct.sizeof(fq.AdamwTensor) == 9 * 8


def test_binding_refuses_host_tensors_and_mismatches():
    x = torch.zeros(4, 8)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        fq.layer_norm(x)
    with pytest.raises(ValueError, match="device"):
        fq.layer_norm_grad(x, x, None, None, torch.zeros(4))
    with pytest.raises(ValueError, match="device"):
        fq.gemm_gated(u8, u8, u8, u8, u8, u8)
    with pytest.raises(ValueError, match="device"):
        fq.adamw_plan([x], [x], [x], [x])
    with pytest.raises(ValueError, match="one entry per tensor"):
        fq.adamw_plan([x], [], [x], [x])
    with pytest.raises(ValueError, match="both or neither"):
        fq.adamw_plan([x], [x], [x], [x], exp_avg_scales=[x])
    with pytest.raises(ValueError, match="8 or 32"):
        fq.adamw_state(x, 4)


def table(L, t, n=None, bits=32, buf=None, nbytes=0):
    arr = (fq.AdamwTensor * max(len(t), 1))(*t)
    size, chunks = ct.c_size_t(nbytes), ct.c_int64(-1)
    status = L.fp4q_adamw_table(arr, len(t) if n is None else n, bits, buf, ct.byref(size), ct.byref(chunks))
    return status, size.value, chunks.value


def test_adamw_table_refusals(L):
    assert table(L, [tensor(), tensor(grad=NUL)])[0] == 1
    assert table(L, [tensor()], n=-1)[0] == 1 and table(L, [tensor()], bits=4)[0] == 1
    assert table(L, [tensor(param=FAKE + 4)])[0] == 3
    arr = (fq.AdamwTensor * 1)(tensor())
    assert L.fp4q_adamw_table(arr, 1, 32, NUL, NUL, NUL) == 1
    status, size, chunks = table(L, [tensor(numel=4096), tensor(numel=4097), tensor(numel=0)])
    assert status == 0 and chunks == 3
    buf = (ct.c_uint8 * (size + 32))()
    at = (ct.addressof(buf) + 15) // 16 * 16
    same = [tensor(numel=4096), tensor(numel=4097), tensor(numel=0)]
    assert table(L, same, buf=at, nbytes=size - 1)[0] == 4
    assert table(L, same, buf=at + 8, nbytes=size)[0] == 3
    assert table(L, same, buf=at, nbytes=size) == (0, size, 3)
    # the owners of the three chunks stand behind the descriptors
    owners = ct.cast(at + size - 12, ct.POINTER(ct.c_uint32))
    assert [owners[i] for i in range(3)] == [0, 1, 1]
    assert table(L, [tensor(numel=(1 << 40) - 1)] * 8)[0] == 2


@pytest.mark.parametrize("kw,status", [
    (dict(table=NUL), 1), (dict(n=-1), 1), (dict(n=0), 1), (dict(chunks=-1), 1), (dict(chunks=1 << 31), 1),
    (dict(table=FAKE + 8), 3), (dict(bits=16), 1), (dict(gdt=3), 1), (dict(lr=-1.0), 1), (dict(step=0), 1),
    (dict(scale=FAKE + 1), 3),
])
def test_adamw_step_table_refusals(L, kw, status):
    a = dict(table=FAKE, n=2, chunks=3, bits=32, gdt=0, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, step=1, seed=0,
             scale=NUL)
    a.update(kw)
    assert L.fp4q_adamw_step_table(*a.values(), NUL) == status
    assert "adamw_step_table" in L.fp4q_last_error().decode()
    assert L.fp4q_adamw_step_table(NUL, 0, 0, 32, 0, 1e-3, 0.9, 0.95, 1e-8, 1, 0, NUL, NUL) == 0


@pytest.mark.parametrize("F", [1, 7])
def test_gated_grad_rows_below_8_elements_have_a_row_limit(L, F):
    """Such rows are 32 to a workgroup of 256 threads, and a launch holds below
    2^32 threads."""
    for M in (1 << 29, (1 << 29) - 31, (1 << 30) - 1):
        assert L.fp4q_gemm_gated_grad(M, F, 64, FAKE, FAKE, FAKE, FAKE, 0, FAKE, FAKE, F, FAKE, FAKE, F,
                                      NUL) == 2
        assert "too many tiles" in L.fp4q_last_error().decode()
