"""Refusals of the residual norms and the gradient norm, on the host: status
codes for every bad argument, nothing launched; what the bindings refuse and
whose memory they hand out."""
import ctypes as ct

import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from test_binding_memory import Dev, MADE, dev, u8, world  # noqa: F401  (world is a fixture)

FAKE = 0x10000   # 16-byte aligned, never dereferenced
NUL = 0
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return fq.lib()


FORWARD = dict(rows=4, cols=64, x=FAKE, xdt=1, ldx=64, b=FAKE, bdt=1, ldb=64, post=0, pw=FAKE, pc=FAKE, gate=FAKE,
               gdt=0, grows=2, ldg=64, xs=1.0, bs=1.0, kind=0, w=FAKE, c=FAKE, wdt=0, eps=1e-5, xo=FAKE, ldxo=64,
               y=FAKE, ydt=1, ldy=64, codes=NUL, scales=NUL, pm=FAKE, pr=FAKE, m=FAKE, r=FAKE)


@pytest.mark.parametrize("kw,status", [
    (dict(x=NUL), 1), (dict(b=NUL), 1), (dict(xo=NUL), 1), (dict(y=NUL), 1), (dict(codes=FAKE), 1),
    (dict(y=NUL, codes=FAKE), 1), (dict(y=NUL, scales=FAKE), 1), (dict(scales=FAKE), 1),
    (dict(xdt=2), 1), (dict(bdt=-1), 1), (dict(wdt=7), 1), (dict(ydt=3), 1), (dict(gdt=3), 1),
    (dict(rows=0), 1), (dict(cols=0), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(cols=1 << 31), 1),
    (dict(ldx=63), 1), (dict(ldb=63), 1), (dict(ldxo=63), 1), (dict(ldy=63), 1), (dict(ldg=63), 1),
    (dict(kind=2), 1), (dict(kind=-1), 1), (dict(post=3), 1), (dict(post=2), 1), (dict(post=2, pw=NUL), 1),
    (dict(grows=0), 1), (dict(grows=-3), 1), (dict(xs=NAN), 1), (dict(bs=INF), 1), (dict(xs=-INF), 1),
    (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(y=NUL, codes=FAKE, scales=FAKE, cols=48), 1),
    (dict(x=FAKE + 1), 3), (dict(b=FAKE + 1), 3), (dict(xo=FAKE + 1), 3), (dict(y=FAKE + 1), 3),
    (dict(pw=FAKE + 2), 3), (dict(pc=FAKE + 2), 3), (dict(w=FAKE + 2), 3), (dict(c=FAKE + 1), 3),
    (dict(gate=FAKE + 2), 3), (dict(pm=FAKE + 2), 3), (dict(pr=FAKE + 1), 3), (dict(m=FAKE + 2), 3),
    (dict(r=FAKE + 2), 3), (dict(y=NUL, codes=FAKE + 8, scales=FAKE), 3),
])
def test_forward_refusals(L, kw, status):
    a = {**FORWARD, **kw}
    assert L.fp4q_residual_norm(*a.values(), NUL) == status
    assert "residual_norm" in L.fp4q_last_error().decode()


BACKWARD = dict(rows=4, cols=64, dy=FAKE, dydt=1, lddy=64, dxo=FAKE, lddxo=64, xo=FAKE, xdt=1, ldxo=64, b=FAKE, bdt=1,
                ldb=64, post=0, pw=FAKE, pc=FAKE, gate=FAKE, gdt=0, grows=2, ldg=64, xs=1.0, bs=1.0, kind=0, w=FAKE,
                wdt=0, pm=FAKE, pr=FAKE, m=FAKE, r=FAKE, dx=FAKE, lddx=64, db=FAKE, lddb=64, dpw=FAKE, dpc=FAKE,
                dg=FAKE, dw=FAKE, dc=FAKE, ws=FAKE, nb=1 << 30)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=NUL), 1), (dict(xo=NUL), 1), (dict(dx=NUL), 1), (dict(db=NUL), 1), (dict(r=NUL), 1), (dict(m=NUL), 1),
    (dict(pm=NUL), 1), (dict(pr=NUL), 1), (dict(post=1, pr=NUL), 1), (dict(b=NUL), 1),
    (dict(b=NUL, post=2, pw=NUL, pc=NUL, dpw=NUL, dpc=NUL), 1), (dict(post=2, pw=NUL, pc=NUL), 1),
    (dict(post=2, pw=NUL, pc=NUL, dpw=NUL), 1), (dict(gate=NUL), 1), (dict(kind=3), 1), (dict(post=-1), 1),
    (dict(dydt=2), 1), (dict(xdt=2), 1), (dict(bdt=5), 1), (dict(gdt=-1), 1), (dict(wdt=2), 1),
    (dict(rows=0), 1), (dict(cols=-4), 1), (dict(rows=1 << 31), 1), (dict(lddy=63), 1), (dict(lddxo=63), 1),
    (dict(ldxo=63), 1), (dict(ldb=63), 1), (dict(ldg=63), 1), (dict(lddx=63), 1), (dict(lddb=63), 1),
    (dict(grows=0), 1), (dict(bs=NAN), 1), (dict(ws=NUL), 1), (dict(ws=FAKE + 8), 3), (dict(nb=64), 4),
    (dict(dy=FAKE + 1), 3), (dict(dxo=FAKE + 1), 3), (dict(xo=FAKE + 1), 3), (dict(b=FAKE + 1), 3),
    (dict(dx=FAKE + 1), 3), (dict(db=FAKE + 1), 3), (dict(dg=FAKE + 2), 3), (dict(dw=FAKE + 2), 3),
    (dict(dpc=FAKE + 1), 3), (dict(pm=FAKE + 2), 3), (dict(w=FAKE + 2), 3), (dict(gate=FAKE + 1), 3),
])
def test_backward_refusals(L, kw, status):
    a = {**BACKWARD, **kw}
    assert L.fp4q_residual_norm_grad(*a.values(), NUL) == status
    assert "residual_norm_grad" in L.fp4q_last_error().decode()


def test_backward_workspace_bytes(L):
    w = L.fp4q_residual_norm_grad_workspace_bytes
    assert w(0, 5, 0) == 0 and w(5, 0, 1) == 0 and w(5, 5, -1) == 0 and w(1, 1, 0) > 0
    assert w(16384, 5120, 0) == w(16384, 5120, 16384) == w(16384, 5120, 1 << 40)
    for each in (0, 1, 2, 63, 64, 65, 1000, 5000, 16383):  # groups of any length
        assert 0 < w(16384, 5120, each) <= 256 << 20
    assert w(100000, 20000, 7) <= 512 << 20  # rows outside the registers


def grads(*t):
    return (fq.Tensor * max(len(t), 1))(*(fq.Tensor(*x) for x in t))


@pytest.mark.parametrize("t,kw,status", [
    ((FAKE, 10, 0), dict(order=2), 1), ((FAKE, 10, 0), dict(max_norm=-1.0), 1), ((FAKE, 10, 0), dict(max_norm=NAN), 1),
    ((FAKE, 10, 0), dict(max_norm=INF), 1), ((FAKE, 10, 0), dict(eps=-1.0), 1), ((FAKE, 10, 0), dict(eps=NAN), 1),
    ((FAKE, 10, 0), dict(n=-1), 1), ((FAKE, 10, 0), dict(norm=NUL, scale=NUL), 1), ((FAKE, 10, 0), dict(ws=NUL), 1),
    ((FAKE, 10, 0), dict(ws=FAKE + 8), 3), ((FAKE, 10, 0), dict(nb=8), 4), ((FAKE, 10, 0), dict(table=FAKE + 8), 3), ((FAKE, 10, 0), dict(norm=FAKE + 2), 3),
    ((FAKE, 10, 0), dict(scale=FAKE + 1), 3), ((NUL, 10, 0), {}, 1), ((FAKE, -1, 0), {}, 1),
    ((FAKE, 1 << 40, 0), {}, 1), ((FAKE, 10, 2), {}, 1), ((FAKE + 2, 10, 0), {}, 3), ((FAKE + 1, 10, 1), {}, 3),
])
def test_grad_norm_refusals(L, t, kw, status):
    a = dict(n=2, table=NUL, order=0, max_norm=1.0, eps=1e-6, norm=FAKE, scale=FAKE, ws=FAKE, nb=1 << 30)
    a.update(kw)
    two = grads((NUL, 0, 0), t)
    assert L.fp4q_grad_norm(two, *a.values(), NUL) == status
    assert "grad_norm" in L.fp4q_last_error().decode()
    if "scale" not in kw:
        a.pop("scale")
        assert L.fp4q_grad_clip(two, *a.values(), NUL) == status
        assert "grad_clip" in L.fp4q_last_error().decode()


def test_grad_scale_refusals_and_empty_calls(L):
    one = grads((FAKE, 10, 0))
    assert L.fp4q_grad_scale(one, 1, NUL, NUL, NUL) == 1
    assert L.fp4q_grad_scale(one, 1, NUL, FAKE + 2, NUL) == 3
    assert L.fp4q_grad_scale(one, 1, FAKE + 4, FAKE, NUL) == 3
    assert L.fp4q_grad_scale(grads((NUL, 10, 0)), 1, NUL, FAKE, NUL) == 1
    assert L.fp4q_grad_scale(NUL, 1, NUL, FAKE, NUL) == 1 and L.fp4q_grad_scale(NUL, -1, NUL, FAKE, NUL) == 1
    assert "grad_scale" in L.fp4q_last_error().decode()
    # nothing to do launches nothing
    assert L.fp4q_grad_scale(NUL, 0, NUL, FAKE, NUL) == 0
    assert L.fp4q_grad_scale(grads(*[(NUL, 0, 1)] * 300), 300, NUL, FAKE, NUL) == 0
    assert L.fp4q_grad_scale(grads(*[(NUL, 0, 1)] * 300), 300, FAKE, FAKE, NUL) == 0
    too_many = grads(*[(FAKE, (1 << 40) - 1, 0)] * 17)
    assert L.fp4q_grad_norm(too_many, 17, NUL, 0, 1.0, 0.0, FAKE, FAKE, FAKE, 1 << 60, NUL) == 2
    assert L.fp4q_grad_norm_workspace_bytes(too_many, 17) == 0
    assert L.fp4q_grad_norm_workspace_bytes(NUL, 0) > 0
    assert ct.sizeof(fq.Tensor) == 24


def table(L, t, buf=NUL, nbytes=0, n=None):
    size = ct.c_size_t(nbytes)
    return L.fp4q_grad_table(grads(*t), len(t) if n is None else n, buf, ct.byref(size)), size.value


def test_grad_table(L):
    assert table(L, [(FAKE, 1, 0), (NUL, 5, 0)])[0] == 1 and table(L, [(FAKE, 1, 0)], n=-1)[0] == 1
    assert table(L, [(FAKE + 2, 1, 0)])[0] == 3 and table(L, [(FAKE, 1, 3)])[0] == 1
    assert L.fp4q_grad_table(grads((FAKE, 1, 0)), 1, NUL, NUL) == 1
    assert table(L, [(FAKE, (1 << 40) - 1, 0)] * 16)[0] == 0
    assert table(L, [(FAKE, (1 << 40) - 1, 0)] * 17)[0] == 2
    same = [(FAKE, 16384, 0), (NUL, 0, 0), (FAKE + 2, 16385, 1), (FAKE, 1, 1)]
    status, size = table(L, same)
    assert status == 0 and size == 4 * 24 + 4 * 4
    buf = (ct.c_uint8 * (size + 32))()
    at = (ct.addressof(buf) + 15) // 16 * 16
    assert table(L, same, at, size - 1)[0] == 4 and table(L, same, at + 8, size)[0] == 3
    assert table(L, same, at, size) == (0, size)
    words = ct.cast(at, ct.POINTER(ct.c_uint64))
    assert [words[i] for i in range(12)] == [FAKE, 16384, 0, 0, 0, 1, FAKE + 2, 16385 | 1 << 62, 1, FAKE,
                                             1 | 1 << 62, 3]
    owners = ct.cast(at + 96, ct.POINTER(ct.c_uint32))
    assert [owners[i] for i in range(4)] == [0, 2, 2, 3]  # the tensor of every 16384 elements


def test_bindings_refuse_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        fq.residual_norm(x, x)
    with pytest.raises(ValueError, match="device"):
        fq.residual_norm_grad(x, x, x, x, (None, None, None, torch.zeros(4)))
    with pytest.raises(ValueError, match="device"):
        fq.grad_plan([x])
    with pytest.raises(ValueError, match="a plan needs"):
        fq.grad_plan([])


@pytest.fixture
def there(world, monkeypatch):  # noqa: F811
    monkeypatch.setattr(Dev, "get_device", lambda self: getattr(self, "at", 0), raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for s in world.values():
        s.device_index = 0
    return world


def rows(*shape, dtype=torch.float32):
    return dev(torch.zeros(shape or (4, 8), dtype=dtype))


def test_bindings_check_shapes_types_and_devices(there):
    x, v = rows(), dev(torch.zeros(8))
    s = dev(torch.zeros(4))
    for kw, e, text in (
            (dict(branch=rows(4, 9)), ValueError, "branch"), (dict(weight=dev(torch.zeros(7))), ValueError, "weight"),
            (dict(weight=v, post_weight=v.bfloat16()), TypeError, "same dtype"),
            (dict(gate=rows(3, 8)), ValueError, "gate_rows is needed"), (dict(gate=rows(2, 7)), ValueError, "gate"),
            (dict(gate=rows(3, 8), gate_rows=3), ValueError, "share one"),
            (dict(gate=rows(2, 8), gate_rows=0), ValueError, "share one"),
            (dict(x_out=rows(4, 8, dtype=torch.bfloat16)), TypeError, "x_out"),
            (dict(y=rows(3, 8)), ValueError, "y must"), (dict(y=rows(), quantize=True), ValueError, "not quantized"),
            (dict(quantize=True), ValueError, "multiple of 32"), (dict(branch=x.expand(2, 4, 8)[0].t()), ValueError, "branch"),
            (dict(branch=dev(torch.zeros(4, 16))[:, ::2]), ValueError, "stride")):
        with pytest.raises(e, match=text):
            fq.residual_norm(x, **{"branch": x, **kw})
    back = dict(dy=x, dx_out=x, x_out=x, branch=x, stats=(None, None, s, s))
    for kw, e, text in (
            (dict(dy=rows(5, 8)), ValueError, "dy"), (dict(dx_out=x.bfloat16()), TypeError, "dx_out"),
            (dict(stats=(None, None, s, dev(torch.zeros(5)))), ValueError, "rstd"),
            (dict(dgate=rows(1, 8)), ValueError, "without a gate"), (dict(want_gate=True), ValueError, "without a gate"),
            (dict(gate=v, dgate=rows(1, 8)), ValueError, "dgate"), (dict(dweight=rows(8, 1)), ValueError, "dweight"),
            (dict(workspace=u8(64)[::2]), ValueError, "contiguous")):
        with pytest.raises(e, match=text):
            fq.residual_norm_grad(**{**back, **kw})
    far = rows()
    far.at = 1
    with pytest.raises(ValueError, match="one device"):
        fq.residual_norm(x, far)
    with pytest.raises(ValueError, match="current device"):
        fq.residual_norm(far, far)
    with pytest.raises(ValueError, match="one device"):
        fq.residual_norm_grad(**{**back, "dy": far})
    with pytest.raises(ValueError, match="one device"):
        fq.grad_plan([x, far])
    there_plan = fq.grad_plan([far])
    there_plan.like.at = 1
    with pytest.raises(ValueError, match="current device"):
        fq.grad_norm(there_plan, 1.0)
    assert all(name.endswith(("_bytes", "_table")) for name, _ in fq._lib.calls)


def test_grad_plan_checks(there):
    for bad, e, text in ((rows(4, 8).half(), TypeError, "bf16 or fp32"), (rows(4, 8)[:, :3], ValueError, "contiguous")):
        with pytest.raises(e, match=text):
            fq.grad_plan([rows(), bad])
    p = fq.grad_plan([rows(), rows(3, 3, dtype=torch.bfloat16), rows(0)])
    assert [(t.numel, t.dtype) for t in p.array] == [(32, 0), (9, 1), (0, 0)]
    for name in ("norm", "scale"):
        with pytest.raises(ValueError, match="one element"):
            fq.grad_norm(p, 1.0, **{name: rows(2)})
    with pytest.raises(ValueError, match="max_norm"):
        fq.grad_norm(p, scale=rows(1))
    with pytest.raises(ValueError, match="one element"):
        fq.scale_grads(p, rows(0))
    with pytest.raises(TypeError, match="scale"):
        fq.scale_grads(p, rows(1).double())
    t = rows()
    p = fq.grad_plan([t])
    t.data = torch.ones(4, 8)
    assert p.tensors[0].data_ptr() == p.array[0].data != t.data_ptr()
    ones = [dev(torch.zeros(8)) for _ in range(2)]
    a = fq.adamw_plan(ones, ones, ones, ones)
    fq.grad_norm(a, 1.0)
    assert fq._lib.calls[-1][1][0] is a.grads.array and a.grads.array[1].data == ones[1].data_ptr()


def test_gradients_that_share_memory_are_not_scaled(there):
    whole = torch.zeros(32)
    part = lambda a, b: dev(whole[a:b])  # noqa: E731
    for grads, shared in (([part(0, 16), part(16, 32), part(16, 16)], False), ([part(16, 32), part(0, 16)], False),
                          ([part(0, 17), part(16, 32)], True), ([part(0, 32), part(4, 5), part(30, 30)], True),
                          ([part(8, 9), part(0, 8), part(8, 9)], True)):
        p = fq.grad_plan(grads)
        fq.grad_norm(p, 1.0)
        for call in (lambda: fq.clip_grads(p, 1.0), lambda: fq.scale_grads(p, rows(1))):
            if shared:
                with pytest.raises(ValueError, match="overlap"):
                    call()
            else:
                call()


def test_what_a_call_allocates_belongs_to_its_stream(there):
    x, s, wide = rows(), dev(torch.zeros(4)), rows(4, 32)
    p = fq.grad_plan([x])
    p.table = u8(64)
    p.table.recorded = set()
    for call, made in ((lambda **kw: fq.residual_norm(x, x, post_kind=fq.LAYER_NORM, **kw), 6),
                       (lambda **kw: fq.residual_norm(wide, wide, quantize=True, kind=fq.RMS_NORM, **kw), 4),
                       (lambda **kw: fq.residual_norm_grad(x, x, x, x, (None, None, s, s), gate=s.new_zeros(8), **kw), 6),
                       (lambda **kw: fq.grad_norm(p, 1.0, **kw), 3), (lambda **kw: fq.clip_grads(p, 1.0, **kw), 2)):
        MADE.clear()
        call(stream=there["side"])
        assert len(MADE) == made
        assert all(t.owner == "side" and "main" in t.recorded for t in MADE)
        assert fq._lib.calls[-1][1][-1] == there["side"].cuda_stream
        MADE.clear()
        call()
        assert len(MADE) == made and all(t.owner == "main" and not t.recorded for t in MADE)
    # the plan's table is read on both, and made on the first
    assert p.table.recorded == {"side"}
