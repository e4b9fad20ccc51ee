"""Which workspace a captured product takes, without a GPU: the capture's state and
the making of workspaces are replaced."""
import pytest
import torch

from weight_only_bit_moe_gb300 import products as P

EAGER, OWN = 1 << 20, 2 << 20
HANDLE = 0x100


@pytest.fixture
def capturing(monkeypatch):
    """Whether the current stream is being captured; it has a workspace already."""
    state = [False]
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: state[0], raising=False)
    monkeypatch.setattr(P, "_captured_workspace", lambda *a: OWN, raising=False)
    monkeypatch.setitem(P._workspaces, (0, HANDLE), (EAGER, None))
    return state


def test_a_captured_call_does_not_share_the_streams_workspace(capturing):
    assert P._workspace(0, HANDLE) == EAGER
    capturing[0] = True
    assert P._workspace(0, HANDLE) == OWN
    capturing[0] = False
    assert P._workspace(0, HANDLE) == EAGER
