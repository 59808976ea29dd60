"""Whose memory the gated, norm and AdamW bindings hand to the kernels, on the
host: the library is replaced by a recorder and device tensors by host ones
that say they are on a device, with a pool that remembers the stream each was
allocated on and recorded on."""
import contextlib

import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq

MADE = []


class Dev(torch.Tensor):
    is_cuda = property(lambda self: True)

    def new_empty(self, size, **kw):
        t = dev(torch.zeros(size, dtype=kw.get("dtype", self.dtype)))
        t.owner, t.recorded = torch.cuda.current_stream().name, set()
        MADE.append(t)
        return t

    def record_stream(self, stream):
        self.recorded.add(stream.name)


class Stream:
    def __init__(self, name, handle):
        self.name, self.cuda_stream = name, handle


def dev(t):
    return t.as_subclass(Dev)


class Recorder:
    """Stands for the library: every call succeeds; remembers the last one."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            self.calls.append((name, a))
            return 64 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def world(monkeypatch):
    MADE.clear()
    streams = dict(main=Stream("main", 0x10), side=Stream("side", 0x20))
    state = dict(now=streams["main"])

    @contextlib.contextmanager
    def stream(s):
        before, state["now"] = state["now"], s
        yield
        state["now"] = before
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state["now"])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: state["now"].cuda_stream)
    monkeypatch.setattr(fq, "_empty_strided_cuda", False)
    monkeypatch.setattr(fq, "_lib", Recorder())
    return streams


def u8(*shape):
    return dev(torch.zeros(shape, dtype=torch.uint8))


def gated(**kw):
    return fq.gemm_gated(u8(4, 64), u8(4, 4), u8(8, 64), u8(8, 4), u8(8, 64), u8(8, 4), save=True, **kw)


def gated_grad(**kw):
    g = dev(torch.zeros(4, 8, dtype=torch.bfloat16))
    return fq.gemm_gated_grad(u8(4, 64), u8(4, 4), u8(8, 64), u8(8, 4), g, g, **kw)


def norm(**kw):
    return fq.layer_norm(dev(torch.zeros(4, 8)), **kw)


def norm_grad(**kw):
    x, s = dev(torch.zeros(4, 8)), dev(torch.zeros(4))
    return fq.layer_norm_grad(x, x, None, s, s, **kw)


@pytest.mark.parametrize("call,made", [(gated, 2), (gated_grad, 1), (norm, 3), (norm_grad, 4)])
def test_what_a_call_allocates_belongs_to_its_stream(world, call, made):
    """Memory from the current stream's pool may still be in use by that
    stream's pending work, and a result that is dropped at once goes back there
    while the other stream's kernel has yet to write it."""
    call(stream=world["side"])
    assert len(MADE) == made
    assert all(t.owner == "side" and "main" in t.recorded for t in MADE)
    assert fq._lib.calls[-1][1][-1] == world["side"].cuda_stream
    MADE.clear()
    call()
    call(stream=world["main"])
    assert len(MADE) == 2 * made
    assert all(t.owner == "main" and not t.recorded for t in MADE)


def plan(n=50, **kw):
    t = [dev(torch.zeros(8)) for _ in range(n)]
    return fq.adamw_plan(t, t, t, t, **kw)


def test_a_plans_table_outlives_the_steps_that_read_it(world, monkeypatch):
    """A step on another stream than the one that made the table still reads it
    when the plan is dropped: the pool has to know of that stream."""
    def tables(*a):
        a[4]._obj.value, a[5]._obj.value = 4096, 50
        return 0
    fq._lib.fp4q_adamw_table = tables
    made = dev(torch.zeros(4096, dtype=torch.uint8))
    made.recorded = set()
    monkeypatch.setattr(torch.Tensor, "to", lambda self, device: made)
    p = plan()
    assert p.table is made
    fq.adamw_step(p, 1e-3, 1)
    fq.adamw_step(p, 1e-3, 1, stream=world["main"])
    assert not made.recorded
    fq.adamw_step(p, 1e-3, 2, stream=world["side"])
    assert made.recorded == {"side"}
    made.recorded.clear()
    p = plan()
    with torch.cuda.stream(world["side"]):
        fq.adamw_step(p, 1e-3, 1)
    assert made.recorded == {"side"}
    assert fq._lib.calls[-1][1][-1] == world["side"].cuda_stream


def test_a_plan_holds_the_memory_it_writes_to(world):
    """A tensor may be given other memory (param.data = ...) behind the plan's
    back: what the plan's addresses name stays allocated all the same."""
    new = [dev(torch.zeros(8)) for _ in range(6)]
    new[5] = new[5].bfloat16()
    p = fq.adamw_plan(*([t] for t in new[:4]), copies=[new[5]])
    for t in new:
        t.data = torch.ones(8, dtype=t.dtype)
    at = p.array[0]
    held = [t for t in p.tensors[0] if t is not None]
    assert [t.data_ptr() for t in held] == [at.param, at.grad, at.exp_avg, at.exp_avg_sq, at.copy]
    assert at.param != new[0].data_ptr()


def test_norm_grad_refuses_workspaces_that_are_not_device_bytes(world):
    """A host workspace, or one whose elements do not lie one behind the other
    (expanded: many elements in the memory of one)."""
    with pytest.raises(ValueError, match="device"):
        norm_grad(workspace=torch.zeros(4096, dtype=torch.uint8))
    for bad in (u8(1).expand(4096), u8(8192)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            norm_grad(workspace=bad)
    assert not fq._lib.calls
    norm_grad(workspace=u8(4096))
    norm_grad(workspace=dev(torch.zeros(32, 32)))
    assert [a[-2] for _, a in fq._lib.calls] == [4096, 4096]


def test_grad_scale_is_one_element(world):
    """Of an empty tensor the address is null, which stands for a scale of 1."""
    p = plan(2)
    for bad in (dev(torch.zeros(0)), dev(torch.ones(2))):
        with pytest.raises(ValueError, match="one element"):
            fq.adamw_step(p, 1e-3, 1, grad_scale=bad)
    assert not fq._lib.calls
    for good in (dev(torch.tensor(0.5)), dev(torch.ones(1))):
        fq.adamw_step(p, 1e-3, 1, grad_scale=good)
        assert fq._lib.calls[-1][1][-2] == good.data_ptr()


def test_dispatch_modes_and_deterministic_fill_see_the_allocations(world, monkeypatch):
    """torch's short way to an allocation passes the dispatcher by; a call goes
    the long way where somebody watches it or wants fresh memory filled."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))
    short = []

    def shortest(size, stride, dtype):
        short.append(size)
        return dev(torch.zeros(size, dtype=dtype))
    monkeypatch.setattr(fq, "_empty_strided_cuda", shortest)
    monkeypatch.setattr(Dev, "get_device", lambda self: 0)
    norm()
    gated()
    assert len(short) == 5 and not MADE
    with Watch():
        norm()
        gated()
    assert len(short) == 5 and len(MADE) == 5
    torch.use_deterministic_algorithms(True)
    try:
        norm()
    finally:
        torch.use_deterministic_algorithms(False)
    assert len(short) == 5 and len(MADE) == 8
    norm()
    assert len(short) == 8
