"""Routing and adapters at the ends of their ranges: rows past 2^31 elements, thousands of
adapters and sequences, sums that the workspace cannot hold in parts."""
import pytest
import torch

from gpu_util import need_gpu
from products_util import offsets_of
from test_gpu_adapters import check_all, make, run_all
from test_gpu_routing import check_balance, check_grad, make_logits
from tuning_util import check_adapter, check_adapter_grads, ref_route

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def A():
    need_gpu()
    from weight_only_bit_moe_gb300 import adapters
    return adapters


@pytest.fixture(scope="module")
def R():
    need_gpu()
    from weight_only_bit_moe_gb300 import routing
    return routing


@pytest.fixture(autouse=True)
def status():
    need_gpu()
    from weight_only_bit_moe_gb300 import products as P
    P.products_status()
    yield
    assert P.products_status() == 0


def spread(t, stride):
    """The matrix with its rows that many elements apart."""
    big = torch.empty(t.shape[0] * stride, dtype=t.dtype, device="cuda")
    view = big.as_strided(t.shape, (stride, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("sizes,rank,n,k", [([200, 93], 16, 136, 264), ([60, 40], 16, 136, 264), ([150, 120], 5, 33, 50)])
def test_rows_far_apart(A, sizes, rank, n, k):
    """Row numbers times strides past 2^31 elements (past 2^32 bytes)."""
    s = make(sizes, rank, n, k, BF, after=7)
    stride = (1 << 32) // sum(sizes) // 8 * 8 + 8  # (a multiple of eight, so that the same kernels run)
    if rank == 5:
        stride += 1
    assert stride * (sum(sizes) - 1) > 2 ** 31
    y, dx, da, db, mid_x, mid_dy = run_all(A, s)
    where = (s["offsets"], s["order"], s["scale"])
    far = spread(s["x"], stride)
    assert torch.equal(A.adapter_mm(far, s["a"], s["b"], *where, base=s["base"]), y)
    assert torch.equal(A.adapter_mm_dw(None, far, None, mid_dy, *where)[0], da)
    del far
    base = spread(s["base"], stride)
    assert A.adapter_mm(s["x"], s["a"], s["b"], *where, base=base, out=base) is base
    assert torch.equal(base, y)
    del base
    far = spread(s["dy"], stride)
    assert torch.equal(A.adapter_mm_dx(far, s["a"], s["b"], *where), dx)
    assert torch.equal(A.adapter_mm_dw(far, None, mid_x, None, *where)[1], db)


@pytest.mark.parametrize("rows", [1, 7, 255, 256, 257, 300])
def test_few_and_many_rows(A, rows):
    """Both sides of the row count where the kernels change."""
    check_all(A, make([rows // 3, 0, rows - rows // 3], 24, 264, 136, BF, before=rows % 2, after=1))


@pytest.mark.parametrize("rank,n,k", [(8, 72, 64), (3, 10, 9)])
@pytest.mark.parametrize("each,rest", [(0, 3), (0, 300), (1, 0)])
def test_thousands_of_adapters(A, rank, n, k, each, rest):
    sizes = [each] * 4096
    sizes[0], sizes[1000], sizes[4095] = 2, 9, 1
    check_all(A, make(sizes, rank, n, k, BF, after=rest))


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_parts_that_the_workspace_does_not_hold(A, dtype):
    check_all(A, make([20000, 77], 256, 64, 72, dtype))   # mid by whole tiles
    check_all(A, make([500, 700], 256, 13000, 12808, dtype))  # gradients by whole adapters


def test_no_rows(A):
    for rank, n, k in ((16, 136, 264), (5, 33, 50)):
        s = make([0, 0], rank, n, k, BF)
        assert A.adapter_mm(s["x"], s["a"], s["b"], s["offsets"], base=s["base"]).shape == (0, n)
        da, db = A.adapter_mm_dw(s["dy"], s["x"], *(torch.zeros(0, rank, device="cuda") for _ in range(2)), s["offsets"])
        assert (da == 0).all() and (db == 0).all() and da.shape == (2, rank, k) and db.shape == (2, n, rank)


@pytest.mark.parametrize("rank", [4, 12])
@pytest.mark.parametrize("sizes", [[1, 0, 2, 61], [100, 180, 40]])
def test_ranks_off_the_grid(A, rank, sizes):
    check_all(A, make(sizes, rank, 264, 520, BF, before=1, after=2), torch.float32)


def test_one_adapter_of_many_rows(A):
    check_all(A, make([70000], 16, 136, 264, BF, order=False))
    check_all(A, make([3, 30000, 5], 40, 264, 136, FP), torch.float32)


def test_mid_alone(A):
    """What the backward pass takes where the rows need no gradient."""
    for sizes in ([3, 4], [150, 200]):
        for rank, n, k in ((16, 136, 264), (5, 33, 50)):
            s = make(sizes, rank, n, k, BF)
            *_, mid_dy = run_all(A, s)
            mid = torch.zeros_like(mid_dy)
            assert A._by_row("moe_adapter_mm_dx", "dy", s["dy"], s["a"], s["b"], s["offsets"], s["order"], s["scale"], None,
                             None, mid, None, False, only_mid=True) is None
            check_adapter(A.adapter_mm_dx(s["dy"], s["a"], s["b"], s["offsets"], s["order"], s["scale"]), mid, s["dy"],
                          s["b"].transpose(1, 2), s["a"].transpose(1, 2), s["offsets"], s["order"], s["scale"], None)


def test_shared_factors(A):
    """One set of factors under several numbers (stride zero)."""
    s = make([40, 0, 90], 16, 136, 200, BF)
    s["a"], s["b"] = s["a"][:1].expand(3, -1, -1), s["b"][:1].expand(3, -1, -1)
    check_all(A, s)


def test_accumulated_twice(A):
    s = make([300, 40], 16, 136, 200, BF)
    *_, mid_x, mid_dy = run_all(A, s)
    where = (s["offsets"], s["order"], s["scale"])
    once = A.adapter_mm_dw(s["dy"], s["x"], mid_x, mid_dy, *where, out_dtype=torch.float32)
    out = tuple(torch.zeros_like(t) for t in once)
    for _ in range(2):
        A.adapter_mm_dw(s["dy"], s["x"], mid_x, mid_dy, *where, out=out, accumulate=True)
    for t, f in zip(out, once):
        assert torch.equal(t, f + f)


# ---------------------------------------------------------------- routing
def test_tokens_far_apart(R):
    logits = make_logits(300, 64)
    far = spread(logits, (1 << 31) // 299 + 1)
    w, ids = R.topk_route(logits, 4)
    got = R.topk_route(far, 4)
    # (rows off the vectors' grid put other experts on a lane: the sums of the weights are the same, of the loss not)
    assert torch.equal(got[1], ids) and torch.allclose(got[0], w, rtol=2.0 ** -20)
    check_grad(R, torch.randn(300, 4, device="cuda"), far, ids, "softmax", False, 1.0)
    check_balance(R, far, R.expert_counts(ids, 64), None, "softmax")


def test_thousands_of_sequences(R):
    lengths = [i % 4 for i in range(3001)]
    logits = make_logits(sum(lengths) + 9, 40)
    ids = R.topk_route(logits, 3)[1]
    offsets = offsets_of(lengths, 4)
    check_balance(R, logits, R.expert_counts(ids, 40, offsets), offsets, "sigmoid")


@pytest.mark.parametrize("lengths", [None, [1000000, 0, 199000]])
def test_a_million_tokens(R, lengths):
    logits = make_logits(1200000, 8)
    ids = R.topk_route(logits, 2)[1]
    want = ref_route(logits, 2, "softmax", None, True, 1.0)[1]
    assert torch.equal(ids, want)
    offsets = None if lengths is None else offsets_of(lengths)
    check_balance(R, logits, R.expert_counts(ids, 8, offsets), offsets, "softmax")


FIRST = """
import torch
from weight_only_bit_moe_gb300 import adapters as A, routing as R, products as P
g = torch.Generator("cuda").manual_seed(0)
sets = []
for dt in (torch.bfloat16, torch.float16):
    for rows in (12, 700):
        for n, k, r in ((50, 44, 5), (72, 64, 8)):
            make = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
            off = torch.tensor([0, rows // 2, rows - 3], dtype=torch.int32, device="cuda")
            sets.append((make(rows, k), make(rows, n), make(2, r, k), make(2, n, r), off))
l, off = torch.randn(700, 64, generator=g, device="cuda"), sets[-1][4]
bias, dloss = torch.zeros(64, device="cuda"), torch.ones(2, device="cuda")
def run():
    out = []
    for x, dy, a, b, o in sets:
        mids = [torch.zeros(x.shape[0], a.shape[1], device="cuda") for _ in range(2)]
        out += [A.adapter_mm(x, a, b, o, mid=mids[0]), A.adapter_mm_dx(dy, a, b, o, mid=mids[1])]
        out += A.adapter_mm_dw(dy, x, *mids, o)
    for top_k in (4, 9):
        w, ids = R.topk_route(l, top_k, "sigmoid", bias)
        out += [w, ids, R.topk_route_grad(w, l, ids, "sigmoid")]
    c = R.expert_counts(ids, 64, off)
    return out + [c, R.balance(l, c, off), R.balance_grad(dloss, l, c, off)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(got, run())) and P.products_status() == 0
"""


def test_first_calls_are_captured(A):
    """A process whose first calls of all these kernels are those of a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
