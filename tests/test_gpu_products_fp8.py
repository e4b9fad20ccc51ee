"""The FP8 block quantisation and the block-scaled FP8 product: codes and scales
bit for bit where the definition fixes them, else against 64 bits."""
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


def normal(*shape, dtype=torch.float32, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ---------------------------------------------------------------- quantisation

def quant_ref(v):
    """The definition on the host, every operation rounded to fp32: v fp32 [rows, K]."""
    v = v.cpu()
    K = v.shape[1]
    pad = torch.nn.functional.pad(v, (0, -K % 128)).unflatten(1, (-1, 128))
    s = torch.clamp_min(pad.abs().amax(2) / 448.0, 2.0 ** -126)
    r = torch.ones_like(s) / s
    q = (pad * r[:, :, None]).flatten(1)[:, :K].to(F8)
    return q, s


def same_codes(q, ref):
    return torch.equal(q.view(torch.uint8).cpu(), ref.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 128), (3, 130), (5, 7), (17, 1024), (64, 2880), (33, 4104), (2, 100),
                                    (700, 512), (1, 7168)])
def test_quant_bit_exact(rows, K, dtype):
    P = products()
    x = (normal(rows, K, seed=1) * torch.exp(2 * normal(K, seed=2))).to(dtype)
    q, s = P.quant_fp8_block(x)
    rq, rs = quant_ref(x.float())
    assert torch.equal(s.cpu(), rs)
    assert same_codes(q, rq)


def test_quant_special_rows():
    P = products()
    x = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = 2.0 ** -133           # the smallest bf16: the scale's floor
    x[2, :] = 3.3e38                # the largest values
    x[3, 200] = float("nan")
    x[4, 5] = float("-inf")
    x[5, :] = -1.0
    x[6, 0], x[6, 1] = 448.0, 2.0 ** -9  # a block whose smallest value is the smallest code
    q, s = P.quant_fp8_block(x)
    rq, rs = quant_ref(x.float())
    for r in (0, 1, 2, 5, 6, 7):
        assert torch.equal(s[r].cpu(), rs[r]) and same_codes(q[r], rq[r])
    v = (q.float() * U.spread_rows(s, 256)).cpu()
    assert not torch.isfinite(v[3, 128:]).any() and (v[3, :128] == 0).all()
    assert not torch.isfinite(v[4, :128]).any() and (v[4, 128:] == 0).all()


def test_quant_gathers_rows():
    P = products()
    x = normal(50, 384, dtype=torch.bfloat16, seed=3)
    rows = torch.tensor([4, 4, 49, 0, -1, 50, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    q, s = P.quant_fp8_block(x, rows=rows)
    src = torch.zeros(8, 384)
    for i, r in enumerate(rows.tolist()):
        if 0 <= r < 50:
            src[i] = x[r].float().cpu()
    rq, rs = quant_ref(src)
    assert torch.equal(s.cpu(), rs) and same_codes(q, rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,K", [(1, 128), (5, 200), (40, 1536), (3, 9), (257, 512)])
def test_quant_gated(rows, K, dtype):
    """|q s - v| is at most half a code step: 2^-4 |v| or s 2^-10 below the normal codes; the fp32 steps before
    the rounding (silu: exponential, sum, quotient, product; the scale and its reciprocal) add 2^-20 |v|."""
    P = products()
    x = (normal(rows, 2 * K, seed=4) * 3).to(dtype)
    q, s = P.quant_fp8_block(x, gated=True)
    g, u = x.double()[:, :K], x.double()[:, K:]
    v = g * torch.sigmoid(g) * u
    top = torch.nn.functional.pad(v, (0, -K % 128)).unflatten(1, (-1, 128)).abs().amax(2) / 448.0
    assert ((s.double() - top).abs() <= 2.0 ** -20 * top).all()
    sw = U.spread_rows(s, K).double()
    err = (q.double() * sw - v).abs()
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, sw * 2.0 ** -10) + 2.0 ** -20 * v.abs()).all()


def test_quant_gate_matches_the_divided_form():
    """Against silu as torch computes it, each operation in fp32 (its exponential and ours differ by a few units
    in the last place at most): q s agrees to half a code step, and the scales to 2^-21."""
    P = products()
    g = torch.linspace(-90, 90, 128 * 64, device="cuda").to(torch.bfloat16).view(64, 128)
    u = torch.full((64, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    q, s = P.quant_fp8_block(torch.cat([g, u], 1), gated=True)
    v = g.float() / (1.0 + torch.exp(-g.float())) * u.float()
    top = (v.abs().amax(1, keepdim=True) / 448.0).clamp_min(2.0 ** -126)
    assert ((s - top).abs() <= 2.0 ** -21 * top + 2.0 ** -120).all()  # (below -87.3 silu is 0)
    err = (q.float() * s - v).abs()
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10) + 2.0 ** -20 * v.abs() + 2.0 ** -110).all()


def test_quant_gate_saturates():
    P = products()
    x = torch.full((2, 256), 1.0, dtype=torch.bfloat16, device="cuda")
    x[0, :128], x[1, :128] = -200.0, 200.0  # exp overflows on one side, vanishes on the other
    q, s = P.quant_fp8_block(x, gated=True)
    v = q.float() * U.spread_rows(s, 128)
    assert (v[0] == 0).all() and ((v[1] - 200).abs() < 1e-3).all()


@pytest.mark.parametrize("pad", [16, 5])
def test_quant_strides(pad):
    P = products()
    x = U.strided(normal(20, 640, dtype=torch.bfloat16, seed=5), pad, float("nan"))
    out = U.strided(torch.zeros(20, 640, device="cuda").to(F8), pad, 0)
    scale = torch.zeros(20, 5, device="cuda")  # row-major scales
    q, s = P.quant_fp8_block(x, out=out, scale=scale)
    assert q is out and s is scale
    rq, rs = quant_ref(x.float())
    assert torch.equal(s.cpu(), rs) and same_codes(q, rq)
    gap = torch.as_strided(out.view(torch.uint8), (19, pad), (640 + pad, 1), 640)
    assert (gap == 0x7F).all()


def test_quant_shifted_base():
    P = products()
    for shift in (1, 2, 4):
        x = normal(9 * 256 + shift, dtype=torch.float16, seed=6)[shift:].view(9, 256)
        out = torch.zeros(9 * 256 + shift, dtype=torch.uint8, device="cuda").view(F8)[shift:].view(9, 256)
        q, s = P.quant_fp8_block(x, out=out)
        rq, rs = quant_ref(x.float())
        assert torch.equal(s.cpu(), rs) and same_codes(q, rq)


# ---------------------------------------------------------------- product

def fp8_case(sizes, N, K, seed, experts):
    rows = sum(sizes)
    P = products()
    x = (normal(rows, K, seed=seed) * torch.exp(normal(K, seed=seed + 1))).to(torch.bfloat16)
    xq, xs = P.quant_fp8_block(x) if rows else (torch.empty(0, K, device="cuda").to(F8),
                                                torch.empty(0, -(-K // 128), device="cuda"))
    wq = (normal(experts, N, K, seed=seed + 2) * 100).clamp(-448, 448).to(F8)
    ws = torch.exp(normal(experts, -(-N // 128), -(-K // 128), seed=seed + 3)) * 1e-3
    return xq, xs, wq, ws


def check_fp8(out, xq, xs, wq, ws, off, K, what=""):
    x, w = xq.double() * U.spread_rows(xs, K).double(), U.dequant_bank(wq, ws)
    for (a, b), ref, mag in U.ref_fwd(x, w, off):
        U.assert_within(out[a:b], ref, mag, K, f"{what} rows {a}:{b}")


FP8_SHAPES = [
    ([1], 16, 16), ([5], 128, 128), ([16, 0, 1, 33], 256, 256), ([64, 63, 65], 200, 144), ([128], 384, 2880),
    ([127, 129, 0, 256, 257], 512, 512), ([300, 1], 1000, 400), ([1000], 264, 1024), ([7] * 30, 136, 272),
    ([2], 4096, 7168), ([700, 40, 900], 1024, 1536), ([0, 1, 2, 5] * 16, 768, 272),
    # more tiles than SMs, and a sum long enough for slices: rows on the M side
    ([127, 129, 0, 256, 257], 2056, 512), ([300, 1, 64] * 4, 1000, 400), ([1000], 1224, 1024), ([300], 2048, 6160),
    # sizes and strides that 16-byte copies cannot address
    ([3], 5, 7), ([40, 0, 70], 130, 129), ([9], 33, 200),
]


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,N,K", FP8_SHAPES, ids=[f"{len(s)}x{sum(s)}-{n}-{k}" for s, n, k in FP8_SHAPES])
def test_fp8_grouped(sizes, N, K, out_dtype):
    P = products()
    xq, xs, wq, ws = fp8_case(sizes, N, K, 10, len(sizes))
    off = U.offsets_of(sizes)
    if out_dtype == torch.float16:
        ws = ws * 1e-2  # inside the type's range
    out = P.gemm_fp8_block(xq, xs, wq, ws, off, out_dtype=out_dtype)
    assert out.dtype == out_dtype
    check_fp8(out, xq, xs, wq, ws, off, K)
    assert torch.equal(P.gemm_fp8_block(xq, xs, wq, ws, off, out_dtype=out_dtype), out)
    assert P.products_status() == 0


@pytest.mark.parametrize("rows", [0, 1, 8, 17, 64, 127, 128, 200, 513])
@pytest.mark.parametrize("N,K", [(512, 640), (72, 2064), (1024, 128)])
def test_fp8_dense(rows, N, K):
    P = products()
    xq, xs, wq, ws = fp8_case([rows], N, K, 20, 1)
    out = P.gemm_fp8_block(xq, xs, wq[0], ws[0])
    assert out.shape == (rows, N)
    check_fp8(out, xq, xs, wq, ws, U.offsets_of([rows]), K)


def test_fp8_rows_of_no_expert():
    P = products()
    xq, xs, wq, ws = fp8_case([150], 256, 384, 30, 2)
    off = torch.tensor([7, 60, 140], dtype=torch.int32, device="cuda")
    xs = xs.clone()
    xs[:7], xs[140:] = float("nan"), float("nan")
    out = torch.full((150, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    P.gemm_fp8_block(xq, xs, wq, ws, off, out=out)
    assert (out[:7] == 9).all() and (out[140:] == 9).all()
    check_fp8(out, xq, xs, wq, ws, off, 384)


@pytest.mark.parametrize("pad", [16, 1])
@pytest.mark.parametrize("rows", [12, 300])
def test_fp8_strides(pad, rows):
    P = products()
    xq, xs, wq, ws = fp8_case([rows], 264, 528, 40, 1)
    x2, w2 = U.strided(xq, pad, 0), U.strided(wq, pad, 0)  # the gaps hold NaN codes
    out = U.strided(torch.zeros(rows, 264, dtype=torch.bfloat16, device="cuda"), pad, 3.0)
    for scale in (xs.contiguous(), xs.t().contiguous().t()):  # row-major and block-major scales
        P.gemm_fp8_block(x2, scale, w2[0], ws[0], out=out)
        check_fp8(out, xq, xs, wq, ws, U.offsets_of([rows]), 528)
    # weight scales read through their strides
    ws2 = ws[0].t().contiguous().t()
    P.gemm_fp8_block(x2, xs, w2[0], ws2, out=out)
    check_fp8(out, xq, xs, wq, ws, U.offsets_of([rows]), 528)
    gap = torch.as_strided(out, (rows - 1, pad), (264 + pad, 1), 264)
    assert (gap == 3.0).all()


def test_fp8_special_values():
    # a NaN row stays in its row, a zero scale gives zeros, negative scales are plain factors
    P = products()
    for rows in (10, 260):
        xq, xs, wq, ws = fp8_case([rows], 256, 256, 50, 1)
        xs, ws = xs.clone(), ws.clone()
        xs[3, 1] = float("nan")
        xs[4] = 0.0
        xs[5] = -xs[5]
        out = P.gemm_fp8_block(xq, xs, wq[0], ws[0])
        assert torch.isnan(out[3]).all() and (out[4] == 0).all()
        keep = [r for r in range(rows) if r != 3]
        x, w = xq.double() * U.spread_rows(xs, 256).double(), U.dequant_bank(wq, ws)
        (_, ref, mag), = U.ref_fwd(x[keep], w, U.offsets_of([rows - 1]))
        U.assert_within(out[keep], ref, mag, 256)


def test_fp8_edges_with_rows_on_m():
    # the three tests above at sizes whose tiles fill the GPU
    P = products()
    xq, xs, wq, ws = fp8_case([150], 5120, 384, 30, 2)
    off = torch.tensor([7, 60, 140], dtype=torch.int32, device="cuda")
    x_scale = xs.clone()
    x_scale[:7], x_scale[140:] = float("nan"), float("nan")
    out = torch.full((150, 5120), 9.0, dtype=torch.bfloat16, device="cuda")
    P.gemm_fp8_block(xq, x_scale, wq, ws, off, out=out)
    assert (out[:7] == 9).all() and (out[140:] == 9).all()
    check_fp8(out, xq, xs, wq, ws, off, 384)

    rows, N, K, pad = 1300, 1000, 528, 16
    xq, xs, wq, ws = fp8_case([rows], N, K, 40, 1)
    x2, w2 = U.strided(xq, pad, 0), U.strided(wq, pad, 0)
    out = U.strided(torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda"), pad, 3.0)
    P.gemm_fp8_block(x2, xs.t().contiguous().t(), w2[0], ws[0].t().contiguous().t(), out=out)
    check_fp8(out, xq, xs, wq, ws, U.offsets_of([rows]), K)
    assert (torch.as_strided(out, (rows - 1, pad), (N + pad, 1), N) == 3.0).all()

    rows = 260
    xq, xs, wq, ws = fp8_case([rows], 4096, 256, 50, 1)
    xs = xs.clone()
    xs[3, 1], xs[4], xs[5] = float("nan"), 0.0, -xs[5]
    out = P.gemm_fp8_block(xq, xs, wq[0], ws[0])
    assert torch.isnan(out[3]).all() and (out[4] == 0).all()
    keep = [r for r in range(rows) if r != 3]
    x, w = xq.double() * U.spread_rows(xs, 256).double(), U.dequant_bank(wq, ws)
    (_, ref, mag), = U.ref_fwd(x[keep], w, U.offsets_of([rows - 1]))
    U.assert_within(out[keep], ref, mag, 256)


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N", [1003, 1016, 977])
def test_fp8_row_ends_inside_a_store(N, out_dtype):
    # rows of the output start on 32 bytes and end anywhere
    P = products()
    rows, K = 1300, 272
    xq, xs, wq, ws = fp8_case([rows], N, K, 70, 1)
    if out_dtype == torch.float16:
        ws = ws * 1e-2
    out = U.strided(torch.zeros(rows, N, dtype=out_dtype, device="cuda"), 1024 - N, 3.0)
    P.gemm_fp8_block(xq, xs, wq[0], ws[0], out=out)
    check_fp8(out, xq, xs, wq, ws, U.offsets_of([rows]), K)
    assert (torch.as_strided(out, (rows - 1, 1024 - N), (1024, 1), N) == 3.0).all()


def test_fp8_offsets_past_32_bits():
    P = products()
    E, N, K = 3, 49152, 49152  # an expert's weights take 2^31.2 bytes
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(F8)
    xq, xs, wq, ws = fp8_case([9, 0, 200], 256, 256, 60, 1)
    w[2, N - 256:, K - 256:] = wq[0]
    scale = torch.ones(E, N // 128, K // 128, device="cuda")
    scale[2, -2:, -2:] = ws[0]
    x = torch.zeros(209, K, device="cuda").to(F8)
    x[:, K - 256:] = xq
    xscale = torch.ones(209, K // 128, device="cuda")
    xscale[:, -2:] = xs
    off = U.offsets_of([9, 0, 200])
    out = P.gemm_fp8_block(x, xscale, w, scale, off)
    assert (out[:9] == 0).all() and (out[9:, :N - 256] == 0).all()
    check_fp8(out[9:, N - 256:], xq[9:], xs[9:], wq, ws, U.offsets_of([200]), 256)
