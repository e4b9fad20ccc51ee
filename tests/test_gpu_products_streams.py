"""Products on several streams and in graphs, with sums cut into slices: the slices
meet in a workspace's counters and partial tiles, so these calls notice one that
is shared, not zeroed or given out again.  Results are compared bit for bit with
those of the same calls made alone."""
import time

import pytest
import torch

from gpu_util import need_gpu
import products_util as U

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def products():
    from weight_only_bit_moe_gb300 import products as P
    return P


class Sliced:
    """Inputs of a decode step's product, an FP8 product of few rows and a gradient of few tiles."""

    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        bf = torch.bfloat16
        self.x, self.w, self.off = normal(5, 4096).to(bf), normal(1, 1024, 4096).to(bf), U.offsets_of([5])
        self.q, self.wq = normal(6, 4096).to(F8), normal(512, 4096).to(F8)
        self.s, self.ws = torch.exp(normal(6, 32)), torch.exp(normal(4, 32))
        self.dy, self.rows, self.at = normal(2500, 264).to(bf), normal(2500, 200).to(bf), U.offsets_of([600, 1900])
        torch.cuda.synchronize()

    def __call__(self, stream=None):
        P = products()
        return [P.grouped_mm(self.x, self.w, self.off, stream=stream),
                P.gemm_fp8_block(self.q, self.s, self.wq, self.ws, stream=stream),
                P.grouped_mm_dw(self.dy, self.rows, self.at, out_dtype=torch.float32, stream=stream)]

    def alone(self):
        out = self()
        torch.cuda.synchronize()
        _, ref, mag = U.ref_fwd(self.x, self.w, self.off)[0]
        U.assert_within(out[0], ref, mag, 4096)
        return out


def same(got, want):
    assert len(got) == len(want)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_two_streams_at_once():
    a, b = Sliced(1), Sliced(2)
    want_a, want_b = a.alone(), b.alone()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    got_a, got_b = [], []
    for _ in range(30):
        got_a.append(a(stream=one))
        got_b.append(b(stream=two))
    torch.cuda.synchronize()
    for ga, gb in zip(got_a, got_b):
        same(ga, want_a)
        same(gb, want_b)


def test_a_replay_beside_calls_on_the_captured_stream():
    P = products()
    a, b = Sliced(3), Sliced(4)
    want_a, want_b = a.alone(), b.alone()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        a()  # the stream has a workspace of its own before the capture
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = a()
    for _ in range(30):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(side):
            got = b()
        side.synchronize()
        other.synchronize()
        same(captured, want_a)
        same(got, want_b)
    assert P.products_status(stream=side) == 0


def test_two_graphs_of_one_stream_at_once():
    a, b = Sliced(5), Sliced(6)
    want_a, want_b = a.alone(), b.alone()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for inputs in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(inputs())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(30):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        same(outs[0], want_a)
        same(outs[1], want_b)


def test_branches_of_a_capture():
    # products on a stream that joined the capture, beside products on the captured one
    P = products()
    a, b = Sliced(7), Sliced(8)
    want_a, want_b = a.alone(), b.alone()
    main, branch = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        branch.wait_stream(main)
        on_branch = [b(stream=branch) for _ in range(3)]
        on_main = [a() for _ in range(3)]
        main.wait_stream(branch)
        after = b()
    graph.replay()
    for _ in range(20):
        for outs in on_branch + on_main + [after]:
            for t in outs:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for outs in on_branch + [after]:
            same(outs, want_b)
        for outs in on_main:
            same(outs, want_a)
    same(a(), want_a)


def test_a_workspace_made_in_a_capture_outlives_it():
    # memory that the graph's own nodes use before is not taken for counters; a graph's end frees its workspace
    P = products()
    a = Sliced(9)
    want = a.alone()

    def capture():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # (dropped: its memory is used again)
            out = a()
            torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        return graph, out

    graph, out = capture()
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)
    torch.cuda.synchronize()
    held = len(P._captured)
    for _ in range(3):
        del graph, out
        torch.cuda.synchronize()
        for _ in range(200):  # (the graph's end is reported from another thread)
            if any(gone.contents.value for _, _, gone in P._captured.values()):
                break
            time.sleep(0.01)
        graph, out = capture()
        assert len(P._captured) <= held
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)


def test_broken_offsets_in_a_replay_are_reported():
    P, B = products(), __import__("weight_only_bit_moe_gb300.binding", fromlist=["binding"])
    a = Sliced(10)
    want = a.alone()
    assert P.products_status() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = a()
    graph.replay()
    assert P.products_status() == 0
    a.off.copy_(U.offsets_of([6]))  # past the rows
    graph.replay()
    a.off.copy_(U.offsets_of([5]))
    graph.replay()  # and right again: what the replay before it found is kept
    assert P.products_status() == B.MOE_ERR_INVALID
    assert P.products_status() == 0
    same(out, want)
    a.off.copy_(U.offsets_of([6]))
    graph.replay()
    torch.cuda.synchronize()
    del graph, out  # nor does the graph's end take it away
    a.off.copy_(U.offsets_of([5]))
    time.sleep(0.2)
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again):
        out = a()
    again.replay()
    assert P.products_status() == B.MOE_ERR_INVALID
    same(out, want)
