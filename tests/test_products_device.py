"""Products whose operands lie on a GPU that is not the current one: the library's
functions launch on the current device, so each call makes the operands' device
current and puts the caller's back.  Runs without a GPU: the tensors claim a
device, the library's functions record which one is current."""
import contextlib

import pytest
import torch

from weight_only_bit_moe_gb300 import products as P

F8 = torch.float8_e4m3fn
HANDLES = {0: 0x100, 1: 0x200}  # each device's current stream
WORKSPACES = {0: 1 << 20, 1: 2 << 20}


class Placed(torch.Tensor):
    """A host tensor that says it lies on GPU 1."""

    def get_device(self):
        return 1


def placed(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=torch.uint8 if dtype is F8 else dtype).view(dtype).as_subclass(Placed)


@pytest.fixture
def calls(monkeypatch):
    """(name, current device, stream handle, workspace or None) of each library call."""
    made, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], torch.device("cuda", index).index if isinstance(index, int) else index.index
        yield
        current[0] = before

    def function(name):
        def fn(*args):
            made.append((name, current[0], args[-1], args[-3] if name != "moe_quant_fp8_block" else None))
            return 0
        return fn

    def status(workspace, stream):
        made.append(("moe_get_status", current[0], stream, workspace))
        return 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: HANDLES[index], raising=False)
    monkeypatch.setattr(P, "_workspace", lambda index, *rest: WORKSPACES[index])
    monkeypatch.setattr(P.B, "function", function)
    monkeypatch.setattr(P.B, "moe_get_status", status)
    yield made
    assert current[0] == 0  # the caller's device is current again


X, W, DY = placed(4, 128), placed(2, 16, 128), placed(4, 16)
OFF = placed(3, dtype=torch.int32)
Q, S = placed(4, 128, dtype=F8), placed(4, 1, dtype=torch.float32)
WQ, WS = placed(2, 16, 128, dtype=F8), placed(2, 1, 1, dtype=torch.float32)

CALLS = {
    "moe_grouped_mm": lambda: P.grouped_mm(X, W, OFF, out=DY),
    "moe_grouped_mm_dx": lambda: P.grouped_mm_dx(DY, W, OFF, out=X),
    "moe_grouped_mm_dw": lambda: P.grouped_mm_dw(DY, X, OFF, out=W),
    "moe_quant_fp8_block": lambda: P.quant_fp8_block(X, out=Q, scale=S),
    "moe_gemm_fp8_block": lambda: P.gemm_fp8_block(Q, S, WQ, WS, OFF, out=DY),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_operands_device_is_current_at_the_launch(calls, name):
    CALLS[name]()
    workspace = None if name == "moe_quant_fp8_block" else WORKSPACES[1]
    assert calls == [(name, 1, HANDLES[1], workspace)]


def test_status_of_another_device(calls):
    assert P.products_status("cuda:1") == 0
    assert P.products_status("cuda") == 0
    assert calls == [("moe_get_status", 1, HANDLES[1], WORKSPACES[1]), ("moe_get_status", 0, HANDLES[0], WORKSPACES[0])]
