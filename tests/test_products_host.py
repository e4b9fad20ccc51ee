"""Refusals of the products (include/moe_products.h) that need no GPU: the C
entries before they touch the device, the PyTorch calls before they call them."""
import pytest
import torch

BUF = 1 << 20  # an address on a 256-byte boundary; nothing reads it


@pytest.fixture(scope="module")
def lib():
    from weight_only_bit_moe_gb300 import build, binding
    build.build()
    return binding


def mm(lib, fn="moe_grouped_mm", **kw):
    a = dict(dtype=0, x=BUF, x_stride=64, w=BUF, w_stride_e=64 * 32, w_stride_n=64, offsets=BUF, num_experts=2,
             rows=10, N=32, K=64, out=BUF, out_stride=64, workspace=BUF,
             workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES, stream=0)
    a.update(kw)
    return getattr(lib.load(), fn)(*a.values())


MM_BAD = [dict(dtype=2), dict(dtype=-1), dict(x_stride=31), dict(w_stride_n=63), dict(out_stride=31),
          dict(w_stride_e=-1), dict(num_experts=0), dict(num_experts=1025), dict(rows=-1), dict(rows=2 ** 31 - 1), dict(N=0), dict(K=0),
          dict(x=0), dict(w=0), dict(offsets=0), dict(out=0), dict(workspace=0), dict(workspace=BUF + 128),
          dict(x=BUF + 1), dict(w=BUF + 1), dict(out=BUF + 1), dict(N=1 << 23)]


@pytest.mark.parametrize("bad", MM_BAD, ids=str)
@pytest.mark.parametrize("fn", ["moe_grouped_mm", "moe_grouped_mm_dx"])
def test_grouped_refusals(lib, fn, bad):
    assert mm(lib, fn, **bad) == lib.MOE_ERR_INVALID


@pytest.mark.parametrize("fn", ["moe_grouped_mm", "moe_grouped_mm_dx"])
def test_grouped_workspace_and_no_rows(lib, fn):
    assert mm(lib, fn, workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES - 1) == lib.MOE_ERR_WORKSPACE
    assert mm(lib, fn, rows=0, x=0, w=0, offsets=0, out=0) == lib.MOE_OK


def dw(lib, **kw):
    a = dict(dtype=0, dy=BUF, dy_stride=32, x=BUF, x_stride=64, offsets=BUF, num_experts=2, rows=10, N=32, K=64,
             dw_dtype=2, accumulate=0, dw=BUF, dw_stride_e=64 * 32, dw_stride_n=64, workspace=BUF,
             workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES, stream=0)
    a.update(kw)
    return lib.load().moe_grouped_mm_dw(*a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dw_dtype=1), dict(dw_dtype=3), dict(accumulate=2), dict(accumulate=1, dw_dtype=0),
    dict(dy_stride=31), dict(x_stride=63), dict(dw_stride_n=63), dict(dw_stride_e=64 * 31 + 63), dict(num_experts=0),
    dict(num_experts=1025), dict(rows=-1), dict(N=0), dict(K=0), dict(dy=0), dict(x=0), dict(offsets=0), dict(dw=0),
    dict(dw=BUF + 2), dict(dy=BUF + 1), dict(workspace=0)], ids=str)
def test_dw_refusals(lib, bad):
    assert dw(lib, **bad) == lib.MOE_ERR_INVALID


def quant(lib, **kw):
    a = dict(dtype=0, x=BUF, x_stride=256, x_rows=4, row_index=0, rows=4, K=128, gated=0, q=BUF, q_stride=128,
             scale=BUF, scale_stride_m=1, scale_stride_g=4, stream=0)
    a.update(kw)
    return lib.load().moe_quant_fp8_block(*a.values())


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(x_stride=127), dict(gated=1, x_stride=255), dict(gated=2), dict(rows=5), dict(rows=-1),
    dict(x_rows=-1), dict(K=0), dict(x=0), dict(q=0), dict(scale=0), dict(q_stride=127), dict(x=BUF + 1)], ids=str)
def test_quant_refusals(lib, bad):
    assert quant(lib, **bad) == lib.MOE_ERR_INVALID


def test_quant_no_rows(lib):
    assert quant(lib, rows=0, x_rows=0, x=0, q=0, scale=0) == lib.MOE_OK


def fp8(lib, **kw):
    a = dict(x=BUF, x_stride=128, x_scale=BUF, xs_m=1, xs_g=4, w=BUF, w_e=0, w_n=128, w_scale=BUF, ws_e=0, ws_n=1,
             ws_k=1, offsets=0, num_experts=1, rows=4, N=64, K=128, out_dtype=0, out=BUF, out_stride=64,
             workspace=BUF, workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES, stream=0)
    a.update(kw)
    return lib.load().moe_gemm_fp8_block(*a.values())


@pytest.mark.parametrize("bad", [
    dict(x_stride=127), dict(w_n=127), dict(out_stride=63), dict(out_dtype=3), dict(out_dtype=-1),
    dict(num_experts=2), dict(num_experts=0), dict(rows=-1), dict(N=0), dict(K=0), dict(x=0), dict(x_scale=0),
    dict(w=0), dict(w_scale=0), dict(out=0), dict(out=BUF + 1), dict(out_dtype=2, out=BUF + 2), dict(workspace=0),
    dict(w_e=-1)], ids=str)
def test_fp8_refusals(lib, bad):
    assert fp8(lib, **bad) == lib.MOE_ERR_INVALID


def test_fp8_no_rows(lib):
    assert fp8(lib, rows=0, x=0, w=0, out=0) == lib.MOE_OK
    assert fp8(lib, workspace_bytes=0) == lib.MOE_ERR_WORKSPACE


def test_python_refusals(lib):
    from weight_only_bit_moe_gb300 import products as P
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 16, 8, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: P.grouped_mm(x, w, off), lambda: P.grouped_mm_dx(x, w, off),
                 lambda: P.grouped_mm_dw(x, x, off), lambda: P.quant_fp8_block(x),
                 lambda: P.gemm_fp8_block(x, x, w, w, off)):
        with pytest.raises(ValueError, match="GPU"):  # no CPU fallback
            call()


@pytest.mark.gpu
def test_python_refusals_on_gpu(lib):
    from gpu_util import need_gpu
    need_gpu()
    from weight_only_bit_moe_gb300 import products as P
    bf, cu = torch.bfloat16, "cuda"
    x, w = torch.zeros(4, 8, dtype=bf, device=cu), torch.zeros(2, 16, 8, dtype=bf, device=cu)
    dy = torch.zeros(4, 16, dtype=bf, device=cu)
    off = torch.zeros(3, dtype=torch.int32, device=cu)
    f8 = torch.float8_e4m3fn
    q, s, wq, ws = x.to(f8), torch.ones(4, 1, device=cu), w.to(f8), torch.ones(2, 1, 1, device=cu)
    bad = [
        lambda: P.grouped_mm(x.float(), w, off),                       # type
        lambda: P.grouped_mm(x.half(), w, off),                        # two types
        lambda: P.grouped_mm(x[:, :7], w, off),                        # width
        lambda: P.grouped_mm(x.t().contiguous().t(), w, off),          # columns apart
        lambda: P.grouped_mm(x[:1].expand(4, 8), w, off),              # rows overlap
        lambda: P.grouped_mm(x, w[0], off),                            # not a bank
        lambda: P.grouped_mm(x, w.transpose(1, 2), off),
        lambda: P.grouped_mm(x, w, off.long()),
        lambda: P.grouped_mm(x, w, off[:2]),
        lambda: P.grouped_mm(x, w, off.cpu()),                         # another device
        lambda: P.grouped_mm(x, w, off, out=dy[:3]),
        lambda: P.grouped_mm(x, w, off, out=dy.float()),
        lambda: P.grouped_mm_dx(x, w, off),
        lambda: P.grouped_mm_dw(dy, x[:3], off),
        lambda: P.grouped_mm_dw(dy, x, off, out_dtype=torch.float16),
        lambda: P.grouped_mm_dw(dy, x, off, accumulate=True),
        lambda: P.grouped_mm_dw(dy, x, off, out=w, accumulate=True),
        lambda: P.grouped_mm_dw(dy, x, off, out=w[:1]),
        lambda: P.quant_fp8_block(x.float()),
        lambda: P.quant_fp8_block(x[:, :7], gated=True),
        lambda: P.quant_fp8_block(x, rows=off.long()),
        lambda: P.quant_fp8_block(x, out=x),
        lambda: P.quant_fp8_block(x, scale=s.half()),
        lambda: P.gemm_fp8_block(x, s, wq, ws, off),
        lambda: P.gemm_fp8_block(q, s[:3], wq, ws, off),
        lambda: P.gemm_fp8_block(q, s, wq, ws[:, :, :0], off),
        lambda: P.gemm_fp8_block(q, s, wq, ws),                        # a bank without offsets
        lambda: P.gemm_fp8_block(q, s, wq, ws, off, out=dy.double()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {i} was accepted")
