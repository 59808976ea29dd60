"""When a gradient plan's table is made, and whose memory it is, on the host."""
import pytest
import torch

import mxfp4_block_scaled_fp4q_amd as fq
from test_abi_residual import rows, there  # noqa: F401  (there is a fixture)
from test_binding_memory import Dev, dev, u8, world  # noqa: F401  (world is a fixture)


@pytest.fixture
def tables(there, monkeypatch):  # noqa: F811
    """The tables that were made, the streams that they belong to, and whether a
    capture is under way."""
    state = dict(made=[], capturing=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])

    def to(self, device):
        t = u8(64)
        t.owner, t.recorded = torch.cuda.current_stream().name, set()
        state["made"].append(t)
        return t
    monkeypatch.setattr(torch.Tensor, "to", to)
    return state


def read():
    """The table that the last call read."""
    name, a = fq._lib.calls[-1]
    assert name in ("fp4q_grad_norm", "fp4q_grad_clip", "fp4q_grad_scale")
    return a[2]


@pytest.mark.parametrize("adamw", [False, True])
def test_a_plan_that_a_capture_left_without_a_table_gets_one(tables, there, adamw):  # noqa: F811
    """No copies inside a capture; the first eager call makes the table, once."""
    t = [dev(torch.zeros(8)) for _ in range(3)]
    plan = fq.adamw_plan(t, t, t, t) if adamw else None
    tables["capturing"] = True
    plan = plan or fq.grad_plan(t)
    for _ in range(2):
        fq.grad_norm(plan, 1.0)
        assert read() is None and not tables["made"]
    tables["capturing"] = False
    fq.grad_norm(plan, 1.0, stream=there["side"])
    (table,) = tables["made"]
    assert read() == table.data_ptr() and table.owner == "main" and table.recorded == {"side"}
    grads = [dev(torch.zeros(8)) for _ in range(2)]
    for call in (lambda: fq.grad_norm(plan, 1.0), lambda: fq.grad_norm(plan, 1.0, stream=there["side"])):
        table.recorded.clear()
        call()
        assert read() == table.data_ptr() and not table.recorded and len(tables["made"]) == 1
    tables["capturing"] = True  # a later capture reads it too
    fq.grad_norm(plan, 1.0)
    assert read() == table.data_ptr() and len(tables["made"]) == 1
    # a plan that was made outside has its table from the start
    tables["capturing"] = False
    with torch.cuda.stream(there["side"]):
        other = fq.grad_plan(grads)
    assert len(tables["made"]) == 2 and other.table.owner == "side"
    fq.clip_grads(other, 1.0)
    assert read() == other.table.data_ptr() and other.table.recorded == {"main"}
    fq.scale_grads(other, rows(1))
    assert read() == other.table.data_ptr()


def test_a_table_belongs_to_its_devices_stream(tables, there, monkeypatch):  # noqa: F811
    """A plan of another device's gradients than the current one's: its memory is
    that device's current stream's, whatever the current device's is called."""
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: (0x10, 0x77)[d])
    monkeypatch.setattr(Dev, "get_device", lambda self: 1)
    plan = fq.grad_plan([dev(torch.zeros(8))])
    (table,) = tables["made"]
    there["side"].device_index, there["side"].cuda_stream = 1, 0x10  # on device 1, not the one it was made on
    plan.read_on(1, there["side"])
    assert table.recorded == {"side"}
    table.recorded.clear()
    there["side"].cuda_stream = 0x77
    plan.read_on(1, there["side"])
    assert not table.recorded
