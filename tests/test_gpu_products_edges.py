"""Values at the ends of fp32's range in the products: small ones in a buffer that a
gradient is added to, scales of opposite size, gates whose exponential nearly
overflows.  Each for operands that the tensor-core kernels take and for others."""
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


def normal(*shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.mark.parametrize("sizes,N,K", [
    ([0, 1900, 0], 264, 200),          # few tiles, sums in slices
    ([0, 40, 0, 0, 300, 0], 1024, 520),
    ([0] * 80 + [3], 512, 256),        # more tiles than CTA pairs
    ([0, 70, 0], 65, 33),              # operands off the 16-byte grid
    ([0, 0], 128, 64),                 # no rows at all
])
def test_accumulation_leaves_experts_without_rows_alone(sizes, N, K):
    """Their gradient is zero, so their part of the buffer keeps its bits: values below fp32's normal range, zeros
    with a sign, infinities and NaN included."""
    P = products()
    dy, x = normal(sum(sizes), N, seed=1).bfloat16(), normal(sum(sizes), K, seed=2).bfloat16()
    start = normal(len(sizes), N, K, seed=3)
    start[:, 1::2] *= 2.0 ** -130
    start[:, 0, 0], start[:, 0, 1], start[:, 0, 2] = -0.0, float("inf"), float("nan")
    out = start.clone()
    P.grouped_mm_dw(dy, x, U.offsets_of(sizes), out=out, accumulate=True)
    for e, m in enumerate(sizes):
        if m == 0:
            assert torch.equal(out[e].view(torch.int32), start[e].view(torch.int32)), f"expert {e}"
        else:
            ref, mag = dy_x(dy, x, sizes, e)
            part = slice(2, None, 2)  # (values that stay in fp32's normal range)
            U.assert_within(out[e][part], (ref + start[e].double())[part], (mag + start[e].double().abs())[part], m + 1)
    assert P.products_status() == 0


def dy_x(dy, x, sizes, e):
    a = sum(sizes[:e])
    d, v = dy[a:a + sizes[e]].double(), x[a:a + sizes[e]].double()
    return d.t() @ v, d.abs().t() @ v.abs()


@pytest.mark.parametrize("rows,N", [(12, 264), (300, 2056)])  # rows on the N and on the M side
@pytest.mark.parametrize("pad", [0, 1])                       # 1: off the 16-byte grid
@pytest.mark.parametrize("up", [120, -120])
def test_fp8_scales_of_opposite_size(rows, N, pad, up):
    """Each block's sum is multiplied by xs * ws: with scales of 2^120 and 2^-120 the result is that of scales of 1,
    although x * xs (up to 2^128.8) or w * ws lies outside fp32."""
    P = products()
    K = 528
    x, w = (normal(rows, K, seed=4) * 150).clamp(-448, 448).to(F8), (normal(N, K, seed=5) * 150).clamp(-448, 448).to(F8)
    xs = torch.full((rows, 5), 2.0 ** up, device="cuda")
    ws = torch.full((-(-N // 128), 5), 2.0 ** -up, device="cuda")
    x, w = (U.strided(t, pad, 0) if pad else t for t in (x, w))
    out = P.gemm_fp8_block(x, xs, w, ws, out_dtype=torch.float32)
    U.assert_within(out, x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t(), K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [512, 130, 200])  # 130: off the 16-byte grid
def test_gates_near_the_exponentials_overflow(dtype, K):
    """silu of -88.69 to -87 in fp32: exp(-g) is finite (up to 88.72), the quotient of the order of 1e-37 and in the
    normal range.  The bounds are those of ordinary gates: half a code step, and 2^-20 for the steps in fp32."""
    P = products()
    g = torch.linspace(-88.6, -87.0, 6 * K, device="cuda").view(6, K).to(dtype)
    g[0, :3] = torch.tensor([-88.5, -88.0, -87.5], device="cuda").to(dtype)
    u = (normal(6, K, seed=6).abs() * 100 + 100).to(dtype)
    q, s = P.quant_fp8_block(torch.cat([g, u], 1), gated=True)
    v = g.double() * torch.sigmoid(g.double()) * u.double()
    top = torch.nn.functional.pad(v, (0, -K % 128)).unflatten(1, (-1, 128)).abs().amax(2) / 448.0
    assert (top > 2.0 ** -126).all()
    assert ((s.double() - top).abs() <= 2.0 ** -20 * top).all()
    sw = U.spread_rows(s, K).double()
    err = (q.double() * sw - v).abs()
    assert (err <= torch.maximum(v.abs() * 2.0 ** -4, sw * 2.0 ** -10) + 2.0 ** -20 * v.abs()).all()


@pytest.mark.parametrize("K", [128, 130])
def test_gated_rows_that_are_not_finite(K):
    """A NaN or an infinity in either half makes its block's values not finite, and no other block's; gates far
    below the overflow give zeros."""
    P = products()
    for value in (float("nan"), float("inf"), float("-inf")):
        for half in (0, 1):
            x = torch.ones(3, 2 * K, dtype=torch.bfloat16, device="cuda")
            x[1, half * K + 5] = value
            x[2, :K] = -100.0
            q, s = P.quant_fp8_block(x, gated=True)
            v = q.float() * U.spread_rows(s, K)
            assert not torch.isfinite(v[1, :128]).any()
            assert torch.isfinite(v[1, 128:]).all() and torch.isfinite(v[0]).all() and (v[0] > 0).all()
            assert (v[2] == 0).all()
