"""The 16-bit products grouped by expert and their gradients against 64-bit
references: ragged and empty groups, sizes around the tiles, both types, row
strides, unaligned operands, rows that no expert has (left alone, and never read:
they hold NaN), gradients against the formula and against differences, autograd,
streams, repeatability and broken offsets."""
import pytest
import torch

from gpu_util import need_gpu
import products_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def products():
    from weight_only_bit_moe_gb300 import products as P
    return P


NAN = float("nan")

# (group sizes, N, K)
SHAPES = [
    ([1], 8, 8),
    ([3], 16, 8),
    ([0, 1, 0, 2, 0], 128, 64),
    ([1, 15, 16, 17, 0, 31, 33], 72, 40),
    ([127, 128, 129, 0, 1], 264, 520),
    ([255, 256, 257], 256, 128),
    ([300, 5, 63, 64, 65], 1000, 712),
    ([513], 512, 1024),
    ([0, 0, 40], 136, 2056),
    ([2000, 1, 700], 384, 320),
    ([0], 64, 64),
    ([7] * 40, 200, 96),
    # operands that 16-byte copies cannot address
    ([1, 2], 7, 5),
    ([70, 0, 33], 65, 33),
    ([9, 130], 129, 100),
]
IDS = [f"{len(s)}x{sum(s)}-{n}-{k}" for s, n, k in SHAPES]


def normal(*shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def check_rows(out, parts, terms, rows, before, what):
    """Rows of the groups against the reference, the others as they were."""
    touched = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for (a, b), ref, mag in parts:
        U.assert_within(out[a:b], ref, mag, terms, f"{what} rows {a}:{b}")
        touched[a:b] = True
    assert torch.equal(out[~touched], before[~touched]), f"{what}: rows of no expert were written"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,N,K", SHAPES, ids=IDS)
def test_fwd(sizes, N, K, dtype):
    P = products()
    rows = sum(sizes) + 12
    off = U.offsets_of(sizes, first=5)
    x, w = normal(rows, K, dtype=dtype, seed=1), normal(len(sizes), N, K, dtype=dtype, seed=2)
    x[:5], x[5 + sum(sizes):] = NAN, NAN
    before = torch.full((rows, N), 7.0, dtype=dtype, device="cuda")
    out = before.clone()
    P.grouped_mm(x, w, off, out=out)
    check_rows(out, U.ref_fwd(x, w, off), K, rows, before, "fwd")
    assert P.products_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,N,K", SHAPES, ids=IDS)
def test_dx(sizes, N, K, dtype):
    P = products()
    rows = sum(sizes) + 12
    off = U.offsets_of(sizes, first=5)
    dy, w = normal(rows, N, dtype=dtype, seed=3), normal(len(sizes), N, K, dtype=dtype, seed=4)
    dy[:5], dy[5 + sum(sizes):] = NAN, NAN
    before = torch.full((rows, K), 7.0, dtype=dtype, device="cuda")
    out = before.clone()
    P.grouped_mm_dx(dy, w, off, out=out)
    check_rows(out, U.ref_dx(dy, w, off), N, rows, before, "dx")
    assert P.products_status() == 0


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                             (torch.float16, torch.float16), (torch.float16, torch.float32)])
@pytest.mark.parametrize("sizes,N,K", SHAPES, ids=IDS)
def test_dw(sizes, N, K, dtype, out_dtype):
    P = products()
    rows = sum(sizes) + 12
    off = U.offsets_of(sizes, first=5)
    dy, x = normal(rows, N, dtype=dtype, seed=5), normal(rows, K, dtype=dtype, seed=6)
    for t in (dy, x):
        t[:5], t[5 + sum(sizes):] = NAN, NAN
    out = P.grouped_mm_dw(dy, x, off, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
        U.assert_within(out[e], ref, mag, m, f"dw expert {e}")
    assert P.products_status() == 0


@pytest.mark.parametrize("sizes,N,K", [SHAPES[i] for i in (2, 4, 9, 13)], ids=[IDS[i] for i in (2, 4, 9, 13)])
def test_dw_accumulate(sizes, N, K):
    P = products()
    off = U.offsets_of(sizes)
    dy = normal(sum(sizes), N, dtype=torch.bfloat16, seed=7)
    x = normal(sum(sizes), K, dtype=torch.bfloat16, seed=8)
    start = normal(len(sizes), N, K, dtype=torch.float32, seed=9)
    out = start.clone()
    assert P.grouped_mm_dw(dy, x, off, out=out, accumulate=True) is out
    for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
        s = start[e].double()
        U.assert_within(out[e], ref + s, mag + s.abs(), m + 1, f"accumulated dw expert {e}")


@pytest.mark.parametrize("sizes", [[2500], [0, 1900, 0], [1500, 40, 1]])
@pytest.mark.parametrize("accumulate", [False, True])
def test_dw_long_sums_over_few_tiles(sizes, accumulate):
    # the rows of an expert are cut into slices, of which a short or empty expert fills few or none
    P = products()
    off = U.offsets_of(sizes)
    N, K = 264, 200
    dy = normal(sum(sizes), N, dtype=torch.bfloat16, seed=40)
    x = normal(sum(sizes), K, dtype=torch.bfloat16, seed=41)
    start = normal(len(sizes), N, K, dtype=torch.float32, seed=42) if accumulate else None
    out = P.grouped_mm_dw(dy, x, off, out=None if start is None else start.clone(), out_dtype=torch.float32,
                          accumulate=accumulate)
    half = P.grouped_mm_dw(dy, x, off)
    for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
        U.assert_within(half[e], ref, mag, m, f"bf16 dw expert {e}")
        if accumulate:
            ref, mag = ref + start[e].double(), mag + start[e].double().abs()
        U.assert_within(out[e], ref, mag, m + 1, f"dw expert {e}")


def test_a_row_of_another_expert_does_not_reach_a_gradient():
    # expert 1's rows, next to expert 0's and 2's last and first, hold NaN and infinities
    P = products()
    sizes = [37, 3, 90]
    off = U.offsets_of(sizes)
    dy = normal(130, 256, dtype=torch.bfloat16, seed=10)
    x = normal(130, 192, dtype=torch.bfloat16, seed=11)
    dy[37:40], x[37:40] = NAN, float("inf")
    out = P.grouped_mm_dw(dy, x, off, out_dtype=torch.float32)
    parts = U.ref_dw(dy, x, off)
    for e in (0, 2):
        U.assert_within(out[e], parts[e][1], parts[e][2], sizes[e], f"expert {e}")
    assert torch.isnan(out[1]).all()
    w = normal(3, 192, 256, dtype=torch.bfloat16, seed=12)
    y = P.grouped_mm(dy, w, off)
    for (a, b), ref, mag in [U.ref_fwd(dy, w, off)[e] for e in (0, 2)]:
        U.assert_within(y[a:b], ref, mag, 256)
    assert torch.isnan(y[37:40]).all()


@pytest.mark.parametrize("pad", [8, 24, 3])  # 3: rows leave the 16-byte grid
def test_row_strides(pad):
    P = products()
    sizes, N, K = [40, 0, 129], 264, 136
    off = U.offsets_of(sizes)
    rows = sum(sizes)
    x = U.strided(normal(rows, K, dtype=torch.bfloat16, seed=13), pad, NAN)
    dy = U.strided(normal(rows, N, dtype=torch.bfloat16, seed=14), pad, NAN)
    w = U.strided(normal(3, N, K, dtype=torch.bfloat16, seed=15), pad, NAN)
    y = U.strided(torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"), pad, 3.0)
    dx = U.strided(torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda"), pad, 3.0)
    dw = U.strided(torch.zeros(3, N, K, dtype=torch.float32, device="cuda"), pad, 3.0)
    P.grouped_mm(x, w, off, out=y)
    P.grouped_mm_dx(dy, w, off, out=dx)
    P.grouped_mm_dw(dy, x, off, out=dw)
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(y[a:b], ref, mag, K, "fwd")
    for (a, b), ref, mag in U.ref_dx(dy, w, off):
        U.assert_within(dx[a:b], ref, mag, N, "dx")
    for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
        U.assert_within(dw[e], ref, mag, m, "dw")
    for t in (y, dx, dw):  # the gaps are as they were
        gap = torch.as_strided(t, (t.numel() // t.shape[-1] - 1, pad), (t.shape[-1] + pad, 1), t.shape[-1])
        assert (gap == 3.0).all()


@pytest.mark.parametrize("shift", [1, 4, 8])  # elements; 8 keeps the 16-byte grid
def test_shifted_bases(shift):
    P = products()
    sizes, N, K = [50, 20], 128, 256
    off = U.offsets_of(sizes)
    flat = normal(70 * K + shift, dtype=torch.float16, seed=16)
    x = flat[shift:].view(70, K)
    w = normal(2 * N * K + shift, dtype=torch.float16, seed=17)[shift:].view(2, N, K)
    out = torch.zeros(70 * N + shift, dtype=torch.float16, device="cuda")[shift:].view(70, N)
    P.grouped_mm(x, w, off, out=out)
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(out[a:b], ref, mag, K, "fwd")


@pytest.mark.parametrize("sizes,N,K", [([2], 1024, 4096), ([1, 0, 5], 128, 8192), ([16] * 8, 1024, 512),
                                       ([900, 300, 0, 4], 2048, 1536), ([64] * 64, 512, 256), ([5000], 640, 768)])
def test_larger_shapes(sizes, N, K):
    # long sums split over CTAs, many experts, more tiles than SMs
    P = products()
    off = U.offsets_of(sizes)
    rows = sum(sizes)
    x, dy = normal(rows, K, dtype=torch.bfloat16, seed=18), normal(rows, N, dtype=torch.bfloat16, seed=19)
    w = normal(len(sizes), N, K, dtype=torch.bfloat16, seed=20)
    y, dx = P.grouped_mm(x, w, off), P.grouped_mm_dx(dy, w, off)
    dw = P.grouped_mm_dw(dy, x, off, out_dtype=torch.float32)
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(y[a:b], ref, mag, K, "fwd")
    for (a, b), ref, mag in U.ref_dx(dy, w, off):
        U.assert_within(dx[a:b], ref, mag, N, "dx")
    for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
        U.assert_within(dw[e], ref, mag, m, "dw")
    for _ in range(3):  # the same inputs give the same bits
        assert torch.equal(P.grouped_mm(x, w, off), y)
        assert torch.equal(P.grouped_mm_dx(dy, w, off), dx)
        assert torch.equal(P.grouped_mm_dw(dy, x, off, out_dtype=torch.float32), dw)
    assert P.products_status() == 0


def test_the_most_experts():
    P = products()
    sizes = [(7 * e) % 5 for e in range(1024)]
    off = U.offsets_of(sizes)
    x, w = normal(sum(sizes), 64, dtype=torch.bfloat16, seed=21), normal(1024, 32, 64, dtype=torch.bfloat16, seed=22)
    y = P.grouped_mm(x, w, off)
    dw = P.grouped_mm_dw(y, x, off, out_dtype=torch.float32)
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(y[a:b], ref, mag, 64)
    for e, (m, ref, mag) in enumerate(U.ref_dw(y, x, off)):
        U.assert_within(dw[e], ref, mag, m)


def test_dw_of_skewed_experts():
    # taken by falling size up to 512 experts, in their order beyond
    P = products()
    for E in (512, 513):
        sizes = [0] * E
        for e in range(E):
            sizes[e] = 700 if e in (3, E - 1) else (e * 5) % 9
        off = U.offsets_of(sizes)
        x, dy = normal(sum(sizes), 40, dtype=torch.bfloat16, seed=49), normal(sum(sizes), 24, dtype=torch.bfloat16, seed=50)
        dw = P.grouped_mm_dw(dy, x, off, out_dtype=torch.float32)
        for e, (m, ref, mag) in enumerate(U.ref_dw(dy, x, off)):
            U.assert_within(dw[e], ref, mag, m, f"expert {e} of {E}")


def test_offsets_past_32_bits():
    # an expert whose weights start more than 2^32 bytes into the bank
    P = products()
    E, N, K = 3, 32768, 32768
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[2, :, :64] = normal(N, 64, dtype=torch.bfloat16, seed=23)
    w[2, N - 1, K - 1] = 2.0
    x = normal(20, K, dtype=torch.bfloat16, seed=24)
    off = U.offsets_of([3, 0, 17])
    y = P.grouped_mm(x, w, off)
    assert (y[:3] == 0).all()
    xe = x[3:].double()
    ref = xe[:, :64] @ w[2, :, :64].double().t()
    mag = xe[:, :64].abs() @ w[2, :, :64].double().abs().t()
    ref[:, N - 1] += 2.0 * xe[:, K - 1]
    mag[:, N - 1] += 2.0 * xe[:, K - 1].abs()
    U.assert_within(y[3:], ref, mag, 65)
    dx = P.grouped_mm_dx(y, w, off)
    yd = y[3:].double()
    assert (dx[3:, 64:K - 1] == 0).all() and (dx[:3] == 0).all()
    U.assert_within(dx[3:, :64], yd @ w[2, :, :64].double(), yd.abs() @ w[2, :, :64].double().abs(), N)
    del w
    dw = P.grouped_mm_dw(y, x, off)
    U.assert_within(dw[2, :, K - 64:], yd.t() @ xe[:, K - 64:], yd.abs().t() @ xe[:, K - 64:].abs(), 17)
    assert (dw[1] == 0).all()


def integers(*shape, top, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(torch.float16)


def test_gradients_against_differences():
    """y is linear in x and in w, so central differences of <dy, y> along a direction equal the gradients'
    products with it; with small whole numbers every product and sum is exact in fp16 (below 2048) and fp32,
    and the two sides are equal."""
    P = products()
    sizes = [19, 0, 45]
    off = U.offsets_of(sizes)
    N, K = 48, 64
    x, w, dy = integers(64, K, top=1, seed=25), integers(3, N, K, top=2, seed=26), integers(64, N, top=1, seed=27)
    dir_x, dir_w = integers(64, K, top=1, seed=28), integers(3, N, K, top=1, seed=29)

    def value(x, w):
        return (dy.double() * P.grouped_mm(x, w, off).double()).sum()

    dx, dw = P.grouped_mm_dx(dy, w, off), P.grouped_mm_dw(dy, x, off)
    assert (value(x + dir_x, w) - value(x - dir_x, w)) / 2 == (dx.double() * dir_x.double()).sum()
    assert (value(x, w + dir_w) - value(x, w - dir_w)) / 2 == (dw.double() * dir_w.double()).sum()


def test_autograd():
    P = products()
    sizes = [10, 0, 54]
    off = U.offsets_of(sizes)
    x = integers(64, 32, top=1, seed=30).requires_grad_()
    w = integers(3, 40, 32, top=1, seed=31).requires_grad_()
    y = P.grouped_linear(x, w, off)
    y.sum().backward()  # the incoming gradient is an expanded scalar
    ones = torch.ones(64, 40, dtype=torch.float16, device="cuda")
    assert torch.equal(x.grad, P.grouped_mm_dx(ones, w.detach(), off))
    assert torch.equal(w.grad, P.grouped_mm_dw(ones, x.detach(), off))
    for (a, b), ref, _ in U.ref_dx(ones, w.detach(), off):
        assert torch.equal(x.grad[a:b].double(), ref)


def test_autograd_with_rows_of_no_expert():
    # experts held elsewhere: their rows come after the last offset
    P = products()
    off = U.offsets_of([7, 20])
    x = integers(40, 16, top=1, seed=47).requires_grad_()
    w = integers(2, 24, 16, top=1, seed=48).requires_grad_()
    y = P.grouped_linear(x, w, off, partial=True)
    assert (y[27:] == 0).all()
    y.square().sum().backward()
    assert (x.grad[27:] == 0).all()
    for (a, b), ref, _ in U.ref_dx(2 * y.detach(), w.detach(), off):
        assert torch.equal(x.grad[a:b].double(), ref)
    for e, (m, ref, _) in enumerate(U.ref_dw(2 * y.detach(), x.detach(), off)):
        assert torch.equal(w.grad[e].double(), ref)


def test_another_stream():
    P = products()
    off = U.offsets_of([100, 28])
    w = normal(2, 256, 512, dtype=torch.bfloat16, seed=32)
    x = normal(128, 512, dtype=torch.bfloat16, seed=33)
    want = P.grouped_mm(x, w, off)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = [P.grouped_mm(x, w, off, stream=st) for _ in range(4)]
    got.append(P.grouped_mm(x, w, off, stream=st.cuda_stream))
    with torch.cuda.stream(st):
        got.append(P.grouped_mm(x, w, off))
    st.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_graph_capture():
    P = products()
    off = U.offsets_of([100, 28])
    w = normal(2, 256, 512, dtype=torch.bfloat16, seed=34)
    x = normal(128, 512, dtype=torch.bfloat16, seed=35)
    out = torch.empty(128, 256, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        P.grouped_mm(x, w, off, out=out)  # the stream's workspace exists before the capture
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        P.grouped_mm(x, w, off, out=out)
    x.copy_(normal(128, 512, dtype=torch.bfloat16, seed=36))
    off.copy_(U.offsets_of([28, 100]))
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(out[a:b], ref, mag, 512)


def test_graph_capture_on_a_stream_of_its_own():
    # a capture on a stream without a workspace takes the graph's memory; long sums use its counters twice
    P = products()
    off = U.offsets_of([5])
    w = normal(1, 1024, 4096, dtype=torch.bfloat16, seed=43)
    x = normal(5, 4096, dtype=torch.bfloat16, seed=44)
    P.grouped_mm(x, w, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = P.grouped_mm(x, w, off)
        second = P.grouped_mm(x, w, off)
    for seed in (45, 46):
        x.copy_(normal(5, 4096, dtype=torch.bfloat16, seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        (_, ref, mag), = U.ref_fwd(x, w, off)
        U.assert_within(first, ref, mag, 4096)
        assert torch.equal(first, second)
    assert torch.equal(P.grouped_mm(x, w, off), first)  # and outside the graph as before


@pytest.mark.parametrize("bad", [[0, 50, 40, 64], [-3, 10, 20, 64], [0, 10, 20, 70]])
def test_broken_offsets_are_reported(bad):
    # they decrease, start below zero or end past the rows: nothing outside the tensors is touched
    P, B = products(), __import__("weight_only_bit_moe_gb300.binding", fromlist=["binding"])
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    base = torch.full((66, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    x, w = normal(64, 64, dtype=torch.bfloat16, seed=37), normal(3, 128, 64, dtype=torch.bfloat16, seed=38)
    P.grouped_mm(x, w, off, out=base[1:65])
    assert P.products_status() == B.MOE_ERR_INVALID
    assert P.products_status() == 0  # read and cleared
    assert (base[0] == 5).all() and (base[65] == 5).all()
    P.grouped_mm_dx(base[1:65], w, off)
    assert P.products_status() == B.MOE_ERR_INVALID
    P.grouped_mm_dw(base[1:65], x, off)
    assert P.products_status() == B.MOE_ERR_INVALID


def test_no_rows():
    P = products()
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    w = normal(2, 16, 24, dtype=torch.bfloat16, seed=39)
    x = torch.empty(0, 24, dtype=torch.bfloat16, device="cuda")
    assert P.grouped_mm(x, w, off).shape == (0, 16)
    dy = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    assert P.grouped_mm_dx(dy, w, off).shape == (0, 24)
    assert torch.equal(P.grouped_mm_dw(dy, x, off), torch.zeros_like(w))


def test_expert_order():
    P = products()
    ids = torch.tensor([[3, 0], [9, 3], [4, 5], [3, 2]], dtype=torch.int32, device="cuda")
    order, off = P.expert_order(ids, 3, expert_base=3)  # this GPU holds experts 3, 4, 5
    assert off.tolist() == [0, 3, 4, 5] and off.dtype == torch.int32
    assert order.tolist()[:5] == [0, 3, 6, 4, 5]
    assert sorted(order.tolist()) == list(range(8))
