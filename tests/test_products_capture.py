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


def test_the_capture_that_counts_is_that_of_the_calls_stream(capturing, monkeypatch):
    captured = set()
    monkeypatch.setattr(P.B, "moe_capture_id", lambda stream: 9 if stream in captured else 0, raising=False)
    capturing[0] = True  # the current stream, but not the one that the call names
    assert P._workspace(0, HANDLE, HANDLE) == EAGER
    capturing[0] = False
    captured.add(HANDLE)
    assert P._workspace(0, HANDLE, HANDLE) == OWN


class Word:
    def __init__(self):
        self.contents = self
        self.value = 0


def test_one_workspace_for_each_stream_of_a_capture(monkeypatch):
    capture, made, words = [1], [], []

    def zeroed(device, ws=None):
        made.append(ws)
        return torch.zeros(16, dtype=torch.uint8) if ws is None else ws

    monkeypatch.setattr(P.B, "moe_capture_id", lambda stream: capture[0], raising=False)
    monkeypatch.setattr(P.B, "moe_capture_watch", lambda stream: words.append(Word()) or words[-1], raising=False)
    monkeypatch.setattr(P, "_zeroed", zeroed, raising=False)
    monkeypatch.setattr(P, "_captured", {}, raising=False)
    first = P._captured_workspace(0, HANDLE)
    assert P._captured_workspace(0, HANDLE) == first and len(made) == 1  # zeroed once
    branch = P._captured_workspace(0, HANDLE + 1)
    capture[0] = 2
    second = P._captured_workspace(0, HANDLE)
    assert len({first, branch, second}) == 3 and made == [None] * 3  # the first graph may still be replayed
    words[0].value = 1
    capture[0] = 3
    assert P._captured_workspace(0, HANDLE) == first  # it is gone, its workspace is zeroed and used again
    assert len(made) == 4 and made[3] is not None


def test_refusals():
    from weight_only_bit_moe_gb300 import build
    build.build()
    B = P.B
    L = B.load()
    assert L.moe_capture_id(None, None) == B.MOE_ERR_INVALID
    assert L.moe_capture_watch(None, None) == B.MOE_ERR_INVALID
    for mode in (-1, 3):
        with pytest.raises(B.MoeError):
            B.moe_capture_mode(mode)


def test_the_status_of_graphs_is_reported(monkeypatch):
    B = P.B
    words = {EAGER: B.MOE_OK, OWN: B.MOE_ERR_INVALID, 3 << 20: B.MOE_ERR_TIMEOUT, 4 << 20: B.MOE_ERR_CUDA}

    def status(workspace, stream):
        word, words[workspace] = words[workspace], B.MOE_OK
        return word

    waited = []
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: HANDLE, raising=False)
    monkeypatch.setattr(torch.cuda, "synchronize", waited.append)
    monkeypatch.setattr(P, "_workspace", lambda *a: EAGER)
    monkeypatch.setattr(P, "_captured", {(0, HANDLE, 1): (OWN, None, Word()), (0, HANDLE, 2): (3 << 20, None, Word()),
                                         (1, HANDLE, 3): (4 << 20, None, Word())}, raising=False)
    monkeypatch.setattr(B, "moe_get_status", status)
    assert P.products_status("cuda:0") == B.MOE_ERR_TIMEOUT and waited == [0]  # (device 1's is not asked for)
    assert P.products_status("cuda:0") == B.MOE_OK  # every word was cleared
    words[OWN] = B.MOE_ERR_INVALID
    assert P.products_status("cuda:0") == B.MOE_ERR_INVALID
