"""Row operands and outputs of more than 2^31 elements, and FP8 experts whose rows are
far from their average, from which the kernel's orientation is chosen."""
import pytest
import torch

from gpu_util import need_gpu
import products_util as U

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
ROWS, WIDE, NARROW, TAIL = 1100003, 2048, 64, 300  # ROWS * WIDE = 2^31.07


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def products():
    from weight_only_bit_moe_gb300 import products as P
    return P


def normal(*shape, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


@pytest.fixture(scope="module")
def wide_rows():
    return torch.cat([normal(100000, WIDE, seed=i).bfloat16() for i in range(11)] + [normal(3, WIDE, seed=11).bfloat16()])


OFF = [0, 700001, ROWS]


def offsets():
    return torch.tensor(OFF, dtype=torch.int32, device="cuda")


def tail_parts(t):
    """The rows around the two experts' border and the last ones, with their expert."""
    return [(slice(OFF[1] - 40, OFF[1]), 0), (slice(OFF[1], OFF[1] + 40), 1), (slice(ROWS - TAIL, ROWS), 1)]


def test_wide_rows_in(wide_rows):
    P, off = products(), offsets()
    w = normal(2, NARROW, WIDE, seed=20).bfloat16()
    y = P.grouped_mm(wide_rows, w, off)
    for s, e in tail_parts(y):
        a, b = wide_rows[s].double(), w[e].double()
        U.assert_within(y[s], a @ b.t(), a.abs() @ b.abs().t(), WIDE)
    dw = P.grouped_mm_dw(y, wide_rows, off, out_dtype=torch.float32)
    ref, mag = torch.zeros(2, NARROW, WIDE, dtype=torch.float64, device="cuda"), torch.zeros_like(dw, dtype=torch.float64)
    for e in range(2):
        for at in range(OFF[e], OFF[e + 1], 100000):
            s = slice(at, min(at + 100000, OFF[e + 1]))
            a, b = y[s].double(), wide_rows[s].double()
            ref[e] += a.t() @ b
            mag[e] += a.abs().t() @ b.abs()
    for e in range(2):
        U.assert_within(dw[e], ref[e], mag[e], OFF[e + 1] - OFF[e])


def test_wide_rows_out():
    P, off = products(), offsets()
    x, w = normal(ROWS, NARROW, seed=21).bfloat16(), normal(2, WIDE, NARROW, seed=22).bfloat16()
    for out, bank in ((P.grouped_mm(x, w, off), w), (P.grouped_mm_dx(x, w.transpose(1, 2).contiguous(), off), w)):
        assert out.numel() > 2 ** 31
        for s, e in tail_parts(out):
            a, b = x[s].double(), bank[e].double()
            U.assert_within(out[s], a @ b.t(), a.abs() @ b.abs().t(), NARROW)


def quant_ref(v):
    pad = v.float().cpu().unflatten(1, (-1, 128))
    s = torch.clamp_min(pad.abs().amax(2) / 448.0, 2.0 ** -126)
    return (pad * (torch.ones_like(s) / s)[:, :, None]).flatten(1).to(F8), s


def test_wide_rows_quantised(wide_rows):
    P = products()
    q, s = P.quant_fp8_block(wide_rows)
    assert q.numel() > 2 ** 31
    back = torch.arange(ROWS - 1, ROWS - 1 - TAIL, -1, dtype=torch.int32, device="cuda")
    gq, gs = P.quant_fp8_block(wide_rows, rows=back)
    rq, rs = quant_ref(wide_rows[-TAIL:])
    assert torch.equal(s[-TAIL:].cpu(), rs) and torch.equal(q[-TAIL:].view(torch.uint8).cpu(), rq.view(torch.uint8))
    assert torch.equal(gs.cpu(), rs.flip(0)) and torch.equal(gq.view(torch.uint8).cpu(), rq.view(torch.uint8).flip(0))
    gated = P.quant_fp8_block(wide_rows, gated=True)
    alone = P.quant_fp8_block(wide_rows[-TAIL:], gated=True)
    for a, b in zip(gated, alone):
        assert torch.equal(a[-TAIL:].view(torch.uint8), b.view(torch.uint8))
    # and on into a product
    wq, ws = normal(NARROW, WIDE, seed=23).to(F8), torch.exp(normal(1, WIDE // 128, seed=24))
    y = P.gemm_fp8_block(q, s, wq, ws)
    a = q[-TAIL:].double() * U.spread_rows(s[-TAIL:], WIDE).double()
    b = U.dequant_bank(wq[None], ws[None])[0]
    U.assert_within(y[-TAIL:], a @ b.t(), a.abs() @ b.abs().t(), WIDE)


@pytest.mark.parametrize("sizes,N,K", [
    ([1500] + [1] * 31, 512, 640),           # one expert has nearly all rows
    ([0] * 20 + [700] + [0] * 11, 384, 1040),
    ([1] * 60 + [0, 900, 0, 3], 2048, 272),
    ([3, 1, 0, 260, 2], 256, 7168),          # a long sum
    ([0, 0, 0, 40], 128, 2880),
])
def test_fp8_experts_far_from_their_average(sizes, N, K):
    P = products()
    E, rows = len(sizes), sum(sizes)
    x, xs = P.quant_fp8_block(normal(rows, K, seed=25).bfloat16())
    w = (normal(E, N, K, seed=26) * 100).clamp(-448, 448).to(F8)
    ws = torch.exp(normal(E, -(-N // 128), -(-K // 128), seed=27)) * 1e-3
    off = U.offsets_of(sizes)
    out = P.gemm_fp8_block(x, xs, w, ws, off)
    for (a, b), ref, mag in U.ref_fwd(x.double() * U.spread_rows(xs, K).double(), U.dequant_bank(w, ws), off):
        U.assert_within(out[a:b], ref, mag, K)
    assert torch.equal(P.gemm_fp8_block(x, xs, w, ws, off), out)
    assert P.products_status() == 0
