"""Low-rank adapters (include/moe_adapters.h) against 64-bit references on the GPU."""
import pytest
import torch

from gpu_util import need_gpu
from products_util import offsets_of
from tuning_util import check_adapter, check_adapter_grads

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def A():
    need_gpu()
    from weight_only_bit_moe_gb300 import adapters
    return adapters


@pytest.fixture(autouse=True)
def status():
    need_gpu()
    from weight_only_bit_moe_gb300 import products as P
    P.products_status()
    yield
    assert P.products_status() == 0


def normal(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def make(sizes, rank, n, k, dtype, order=True, before=0, after=0, seed=0, scale=True, base=True):
    gen = torch.Generator("cuda").manual_seed(seed)
    rows, L = before + sum(sizes) + after, len(sizes)
    s = dict(x=normal(gen, rows, k, dtype=dtype), a=normal(gen, L, rank, k, dtype=dtype, scale=k ** -0.5),
             b=normal(gen, L, n, rank, dtype=dtype, scale=rank ** -0.5), dy=normal(gen, rows, n, dtype=dtype),
             offsets=offsets_of(sizes, before), order=None,
             scale=normal(gen, L) + 1.5 if scale else None, base=normal(gen, rows, n, dtype=dtype) if base else None)
    if order:
        s["order"] = torch.randperm(rows, generator=gen, device="cuda").to(torch.int32)
    return s


def run_all(A, s, out_dtype=None):
    rows, rank = s["x"].shape[0], s["a"].shape[1]
    mid_x, mid_dy = (torch.full((rows, rank), float("nan"), device="cuda") for _ in range(2))
    where = (s["offsets"], s["order"], s["scale"])
    y = A.adapter_mm(s["x"], s["a"], s["b"], *where, base=s["base"], mid=mid_x)
    dx = A.adapter_mm_dx(s["dy"], s["a"], s["b"], *where, mid=mid_dy)
    da, db = A.adapter_mm_dw(s["dy"], s["x"], mid_x, mid_dy, *where, out_dtype=out_dtype)
    return y, dx, da, db, mid_x, mid_dy


def check_all(A, s, out_dtype=None):
    y, dx, da, db, mid_x, mid_dy = run_all(A, s, out_dtype)
    where = (s["offsets"], s["order"], s["scale"])
    check_adapter(y, mid_x, s["x"], s["a"], s["b"], *where, s["base"], "y")
    check_adapter(dx, mid_dy, s["dy"], s["b"].transpose(1, 2), s["a"].transpose(1, 2), *where, None, "dx")
    check_adapter_grads(da, db, s["dy"], s["x"], mid_x, mid_dy, *where, what="")


SIZES = [
    ([1], 16, 1024, 512),                        # one token
    ([1, 0, 1, 2, 0, 1], 16, 512, 1024),         # decode: a row or two each, adapters without rows
    ([0, 0], 8, 64, 64),                         # no rows at all
    ([17, 130, 0, 1, 64], 8, 264, 200),          # ragged
    ([127, 128, 129], 32, 320, 384),             # around a tile
    ([300], 64, 512, 520),
    ([5, 255, 257], 128, 256, 768),
    ([40, 200], 256, 136, 328),                  # the largest rank
    ([33, 70], 24, 1000, 72),
    ([9, 100], 40, 8, 8),                        # narrow
    ([1] * 70, 16, 256, 2880),                   # a batch of requests, each with its own
    ([700, 650], 16, 2880, 640),
]
ODD = [
    ([3, 0, 66], 3, 13, 7),                      # off every grid
    ([2, 5], 1, 1, 1),
    ([70, 1], 17, 129, 65),
    ([65], 12, 100, 36),                         # multiples of four
    ([20, 30], 255, 33, 31),
]


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(SIZES + ODD)))
def test_sizes(A, case, dtype):
    sizes, rank, n, k = (SIZES + ODD)[case]
    check_all(A, make(sizes, rank, n, k, dtype, before=2 * (case % 2), after=case % 3, seed=case))


@pytest.mark.parametrize("order", [True, False])
@pytest.mark.parametrize("scale,base", [(True, False), (False, True)])
def test_without_order_scale_or_base(A, order, scale, base):
    for sizes, rank, n, k in (([30, 0, 150], 16, 264, 328), ([4, 9], 5, 20, 30)):
        check_all(A, make(sizes, rank, n, k, BF, order=order, before=3, after=5, scale=scale, base=base), torch.float32)


@pytest.mark.parametrize("rank,n,k", [(16, 264, 328), (6, 50, 44)])
def test_in_place_leaves_other_rows(A, rank, n, k):
    s = make([20, 130], rank, n, k, BF, before=7, after=9)
    want = A.adapter_mm(s["x"], s["a"], s["b"], s["offsets"], s["order"], s["scale"], base=s["base"])
    y = s["base"].clone()
    for r in s["order"][torch.tensor([0, 6, 157, 165], device="cuda")].tolist():
        y[r] = float("nan")  # (not read: the bits stay)
    before = y.clone()
    assert A.adapter_mm(s["x"], s["a"], s["b"], s["offsets"], s["order"], s["scale"], base=y, out=y) is y
    rows = s["order"][7:157].long()
    assert torch.equal(y[rows], want[rows])
    others = torch.cat([s["order"][:7], s["order"][157:]]).long()
    assert torch.equal(y[others].view(torch.int16), before[others].view(torch.int16))


@pytest.mark.parametrize("rank,n,k,pad", [(16, 264, 328, 8), (32, 136, 72, 16), (5, 50, 44, 3), (8, 64, 64, 1)])
def test_strides_and_what_lies_around(A, rank, n, k, pad):
    """Operands inside larger buffers of NaN; outputs inside buffers whose rest keeps its bits."""
    s = make([20, 130, 3], rank, n, k, BF, before=1, after=2)

    def inside(t):
        big = torch.full((t.shape[0] + 2, *t.shape[1:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype, device="cuda")
        view = big[1:-1, ..., :t.shape[-1]]
        view.copy_(t)
        return view

    y, dx, da, db, mid_x, mid_dy = run_all(A, s)
    v = {key: inside(s[key]) if key in ("x", "a", "b", "dy", "base") else s[key] for key in s}
    where = (s["offsets"], s["order"], s["scale"])
    outs = [inside(torch.zeros_like(t)) for t in (y, dx, da, db)]
    A.adapter_mm(v["x"], v["a"], v["b"], *where, base=v["base"], out=outs[0])
    A.adapter_mm_dx(v["dy"], v["a"], v["b"], *where, out=outs[1])
    A.adapter_mm_dw(v["dy"], v["x"], mid_x, mid_dy, *where, out=(outs[2], outs[3]))
    check_adapter(outs[0], None, s["x"], s["a"], s["b"], *where, s["base"], "y")
    check_adapter(outs[1], None, s["dy"], s["b"].transpose(1, 2), s["a"].transpose(1, 2), *where, None, "dx")
    check_adapter_grads(outs[2], outs[3], s["dy"], s["x"], mid_x, mid_dy, *where)
    for t in outs:
        big = t._base
        assert torch.isnan(big[0]).all() and torch.isnan(big[-1]).all() and torch.isnan(big[..., t.shape[-1]:]).all()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("rank,n,k", [(16, 264, 328), (5, 50, 44)])
def test_rows_do_not_meet(A, rank, n, k, dtype):
    """A NaN or an infinity in one adapter's rows or factors stays with that adapter."""
    s = make([9, 50, 70], rank, n, k, dtype, after=4)
    clean = run_all(A, s)
    first = s["order"][:9].long()
    s["x"][first], s["dy"][first] = float("inf"), float("nan")
    s["x"][s["order"][-1].long()] = float("nan")
    s["a"][0, 0, 0] = float("nan")
    got = run_all(A, s)
    rest = s["order"][9:].long()
    for i in (0, 1):
        assert torch.equal(got[i][rest], clean[i][rest])
    for i in (2, 3):
        assert torch.equal(got[i][1:], clean[i][1:])
    assert not torch.isfinite(got[0][first]).any()


def test_same_bits_twice(A):
    for sizes, rank, n, k in (([200, 311], 32, 520, 1032), ([1] * 40, 16, 1024, 2048), ([30, 9], 7, 33, 41)):
        s = make(sizes, rank, n, k, BF)
        for a, b in zip(run_all(A, s)[:4], run_all(A, s)[:4]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rank,n,k", [(16, 264, 328), (5, 50, 44)])
def test_accumulated_gradients(A, rank, n, k):
    s = make([40, 0, 200], rank, n, k, BF, after=3)
    _, _, _, _, mid_x, mid_dy = run_all(A, s)
    gen = torch.Generator("cuda").manual_seed(5)
    start = normal(gen, 3, rank, k), normal(gen, 3, n, rank)
    start[0][1, 0, 0] = float("nan")  # (an adapter without rows keeps its bits)
    out = tuple(t.clone() for t in start)
    got = A.adapter_mm_dw(s["dy"], s["x"], mid_x, mid_dy, s["offsets"], s["order"], s["scale"], out=out, accumulate=True)
    assert got[0] is out[0] and got[1] is out[1]
    for t, f in zip(out, start):
        assert torch.equal(t[1].view(torch.int32), f[1].view(torch.int32))
    keep = [0, 2]
    for l in keep:
        two = s["offsets"][l:l + 2]
        c = s["scale"][l:l + 1]
        check_adapter_grads(out[0][l:l + 1], out[1][l:l + 1], s["dy"], s["x"], mid_x, mid_dy, two, s["order"], c,
                            (start[0][l:l + 1], start[1][l:l + 1]))


def test_one_gradient_alone(A):
    for rank in (16, 6):
        s = make([40, 90], rank, 264, 328, FP)
        _, _, da, db, mid_x, mid_dy = run_all(A, s)
        where = (s["offsets"], s["order"], s["scale"])
        only_a = A.adapter_mm_dw(None, s["x"], None, mid_dy, *where)
        only_b = A.adapter_mm_dw(s["dy"], None, mid_x, None, *where)
        assert only_a[1] is None and torch.equal(only_a[0], da)
        assert only_b[0] is None and torch.equal(only_b[1], db)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
def test_magnitudes_far_apart(A, dtype):
    """Rows whose mids differ by many powers of two, and factors near the type's ends."""
    s = make([64, 64], 16, 128, 256, dtype, scale=False, base=False)
    small, large = (2.0 ** -20, 2.0 ** 20) if dtype is BF else (2.0 ** -8, 2.0 ** 8)
    at = s["order"].long()
    s["x"][at[::2]] = (s["x"][at[::2]].float() * small).to(dtype)
    s["dy"][at[1::3]] = (s["dy"][at[1::3]].float() * small).to(dtype)
    s["b"] = (s["b"].float() * large ** 0.5).to(dtype)
    check_all(A, s, torch.float32)


def test_mid_larger_than_the_workspace(A):
    """Past the rows whose mids the workspace keeps."""
    rows = (1 << 22) // 64 + 77
    s = make([rows - 5], 64, 16, 24, BF, order=False, after=5)
    got = A.adapter_mm(s["x"], s["a"], s["b"], s["offsets"], None, s["scale"], base=s["base"])
    check_adapter(got, None, s["x"], s["a"], s["b"], s["offsets"], None, s["scale"], s["base"])


@pytest.mark.parametrize("rank,n,k", [(16, 264, 328), (5, 50, 44)])
def test_broken_offsets_and_orders_are_reported(A, rank, n, k):
    from weight_only_bit_moe_gb300 import products as P
    s = make([20, 130, 3], rank, n, k, BF, after=2)
    good = s["offsets"].clone()

    def bad(offsets=None, order=None):
        offsets, order = s["offsets"] if offsets is None else offsets, s["order"] if order is None else order
        mid_x, mid_dy = (torch.zeros(155, rank, device="cuda") for _ in range(2))
        for call in (lambda: A.adapter_mm(s["x"], s["a"], s["b"], offsets, order, base=s["base"], mid=mid_x),
                     lambda: A.adapter_mm_dx(s["dy"], s["a"], s["b"], offsets, order, mid=mid_dy),
                     lambda: A.adapter_mm_dw(s["dy"], s["x"], mid_x, mid_dy, offsets, order)):
            call()
            assert P.products_status() == P.B.MOE_ERR_INVALID

    for at, value in ((0, -5), (1, 151), (2, 3), (3, 10 ** 6), (3, -1)):
        broken = good.clone()
        broken[at] = value
        bad(offsets=broken)
    for value in (-1, 155, 2 ** 31 - 1, -2 ** 31):
        broken = s["order"].clone()
        broken[40] = value
        bad(order=broken)
    check_all(A, s)


# ---------------------------------------------------------------- gradients
@pytest.mark.parametrize("order", [True, False])
def test_autograd(A, order):
    s = make([40, 0, 90], 16, 136, 200, BF, order=order, after=6)
    leaves = [s[key].clone().requires_grad_() for key in ("x", "a", "b", "base")]
    y = A.adapter_linear(*leaves[:3], s["offsets"], s["order"], s["scale"], base=leaves[3])
    grads = torch.autograd.grad(y, leaves, s["dy"])
    want_y, dx, da, db, _, _ = run_all(A, s)
    for got, want in zip((y, *grads), (want_y, dx, da, db, s["dy"])):
        assert torch.equal(got, want)
    # each alone, and gradients that arrive in strides of their own
    for i in range(4):
        only = [t.detach().requires_grad_(i == j) for j, t in enumerate(leaves)]
        y = A.adapter_linear(*only[:3], s["offsets"], s["order"], s["scale"], base=only[3])
        g = torch.autograd.grad(y, only[i], s["dy"].t().contiguous().t())[0]
        assert torch.equal(g, grads[i])
    with pytest.raises(RuntimeError):  # no second derivatives
        y = A.adapter_linear(*leaves[:3], s["offsets"], s["order"], s["scale"])
        g = torch.autograd.grad(y, leaves[0], s["dy"], create_graph=True)[0]
        torch.autograd.grad(g.sum(), leaves[1])


@pytest.mark.parametrize("which", ["x", "a", "b"])
def test_gradients_against_differences(A, which):
    """The product is linear in each argument: <dy, f(v + d) - f(v - d)> / 2 = <gradient, d> for any d."""
    s = make([40, 90], 16, 136, 200, FP, base=False)
    gen = torch.Generator("cuda").manual_seed(9)
    v = s[which]
    d = (normal(gen, *v.shape) * v.float().abs().mean()).to(FP)
    up, down = (v.float() + d.float()).to(FP), (v.float() - d.float()).to(FP)
    step = (up.double() - down.double()) / 2
    f = [A.adapter_mm(*(t if key == which else s[key] for key in ("x", "a", "b")), s["offsets"], s["order"], s["scale"])
         for t in (up, down)]
    leaf = ((up.double() + down.double()) / 2).to(FP).requires_grad_()
    y = A.adapter_linear(*(leaf if key == which else s[key] for key in ("x", "a", "b")), s["offsets"], s["order"],
                         s["scale"])
    g = torch.autograd.grad(y, leaf, s["dy"])[0].double()
    left = (s["dy"].double() * (f[0].double() - f[1].double())).sum() / 2
    right = (g * step).sum()
    # outputs and gradient are rounded to 11 bits, with their sums' and mids' 2^-16 beside
    bound = 2.0 ** -10 * ((s["dy"].double().abs() * (f[0].double().abs() + f[1].double().abs())).sum() / 2
                          + (g.abs() * step.abs()).sum())
    assert abs(left - right) <= bound
    assert abs(right) > 4 * 2.0 ** -10 * right.abs().clamp_min(1e-9)  # (a direction that counts)


# ---------------------------------------------------------------- streams and graphs
def test_on_another_stream(A):
    s = make([40, 90], 16, 264, 328, BF)
    want = run_all(A, s)
    side = torch.cuda.Stream()
    where = (s["offsets"], s["order"], s["scale"])
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y = A.adapter_mm(s["x"], s["a"], s["b"], *where, base=s["base"], stream=stream)
        dx = A.adapter_mm_dx(s["dy"], s["a"], s["b"], *where, stream=stream)
        da, db = A.adapter_mm_dw(s["dy"], s["x"], want[4], want[5], *where, stream=stream)
        side.synchronize()
        for got, ref in zip((y, dx, da, db), want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("sizes", [[1] * 12, [40, 90, 200]])
def test_captured_and_replayed(A, sizes):
    s = make(sizes, 16, 264, 328, BF)
    run_all(A, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_all(A, s)
    other = make(sizes, 16, 264, 328, BF, seed=3)
    want = run_all(A, other)
    for key in ("x", "a", "b", "dy", "base", "order", "scale"):
        s[key].copy_(other[key])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got[:4], want):
        assert torch.equal(a, b)


def test_beside_a_captured_one(A):
    """A replay and eager calls at one time, on two streams."""
    s, other = make([300, 290], 32, 520, 1032, BF), make([300, 290], 32, 520, 1032, BF, seed=3)
    want, want_other = run_all(A, s), run_all(A, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_all(A, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = []
    for _ in range(5):
        with torch.cuda.stream(side):
            graph.replay()
        eager.append(run_all(A, other))
    torch.cuda.synchronize()
    for a, b in zip(got[:4], want):
        assert torch.equal(a, b)
    for e in eager:
        for a, b in zip(e[:4], want_other):
            assert torch.equal(a, b)
