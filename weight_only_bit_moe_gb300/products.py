"""PyTorch-facing calls of the products in include/moe_products.h: 16-bit products
grouped by expert with their gradients, and the FP8 product with block scales with
the quantisation that feeds it.  Like ``layer`` they own buffers and check
arguments; the arithmetic runs in the library's kernels.

Rows of one expert are consecutive; ``offsets`` (int32, [E + 1], on the device)
says where each expert's rows start.  ``expert_order`` makes both from routing ids::

    order, offsets = expert_order(topk_ids, E)        # order[i]: pair of row i
    h = grouped_linear(x[order // top_k], w, offsets)  # differentiable

    q, s = quant_fp8_block(x, rows=order // top_k)     # gathered on the way
    h = gemm_fp8_block(q, s, w_fp8, w_scale, offsets)
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B

BLOCK = 128  # columns per FP8 scale; also rows of a weight block
_DTYPE = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16, torch.float32: B.MOE_FP32}
_HALF = (torch.bfloat16, torch.float16)

# One workspace per device and stream, as the kernels of one stream run one after another.
_workspaces = {}


def _handle(device: torch.device, stream) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(device: torch.device, handle: int) -> torch.Tensor:
    ws = _workspaces.get((device.index, handle))
    if ws is None:
        ws = torch.zeros(B.MOE_PRODUCTS_WORKSPACE_BYTES, dtype=torch.uint8, device=device)
        # the zeros are written on the current stream, the kernels run on `handle`
        torch.cuda.current_stream(device).synchronize()
        _workspaces[(device.index, handle)] = ws
    return ws


def products_status(device="cuda", stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status of its products:
    MOE_OK, MOE_ERR_TIMEOUT or MOE_ERR_INVALID (offsets that decrease or leave the rows)."""
    device = torch.device("cuda", torch.cuda.current_device()) if str(device) == "cuda" else torch.device(device)
    handle = _handle(device, stream)
    return B.moe_get_status(_workspace(device, handle), handle)


def _matrix(t: torch.Tensor, name: str, width: Optional[int] = None, rows: Optional[int] = None) -> int:
    """Row stride of a 2-D row-major matrix of `width` columns."""
    if t.dim() != 2 or (width is not None and t.shape[1] != width) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [{'rows' if rows is None else rows}, "
                         f"{'columns' if width is None else width}]")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous (strides {t.stride()})")
    if t.shape[0] <= 1:
        return max(t.stride(0), t.shape[1])
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return t.stride(0)


def _bank(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(expert, row) strides of a bank [E, N, K]."""
    if t.dim() != 3:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [experts, N, K]")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous (strides {t.stride()})")
    row = t.stride(1) if t.shape[1] > 1 else max(t.stride(1), t.shape[2])
    if row < t.shape[2]:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return t.stride(0), row


def _on(device: torch.device, **tensors) -> None:
    if device.type != "cuda":
        raise ValueError(f"the products run on a GPU, not on {device}")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _check_offsets(offsets: torch.Tensor, E: int) -> None:
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.shape[0] != E + 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets: expected contiguous int32 [{E + 1}], got {offsets.dtype} {tuple(offsets.shape)}")


def _half(name: str, *tensors: torch.Tensor) -> int:
    dtype = tensors[0].dtype
    if dtype not in _HALF or any(t.dtype != dtype for t in tensors):
        raise ValueError(f"{name}: operands of one type, bfloat16 or float16, expected; got "
                         f"{', '.join(str(t.dtype) for t in tensors)}")
    return _DTYPE[dtype]


def expert_order(topk_ids: torch.Tensor, num_experts: int, expert_base: int = 0):
    """(order, offsets) of routing ids [M, top_k]: order int32 holds the pairs (token * top_k + slot) by
    expert, in pair order within one, and offsets int32 [num_experts + 1] each expert's first row.  Pairs of
    experts held elsewhere come after offsets[num_experts]."""
    ids = topk_ids.reshape(-1).to(torch.int64) - expert_base
    ids = torch.where((ids >= 0) & (ids < num_experts), ids, num_experts)
    order = torch.sort(ids, stable=True).indices.to(torch.int32)
    counts = torch.zeros(num_experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(
        0, ids, torch.ones_like(ids))
    offsets = torch.zeros(num_experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, 0)[:num_experts]
    return order, offsets


def grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows r of expert e: x [rows, K], w [E, N, K] -> [rows, N]."""
    dev = x.device
    _on(dev, w=w, offsets=offsets, out=out)
    w_e, w_n = _bank(w, "w")
    E, N, K = w.shape
    ld = _matrix(x, "x", K)
    _check_offsets(offsets, E)
    if out is None:
        out = torch.empty((x.shape[0], N), dtype=x.dtype, device=dev)
    dt = _half("grouped_mm", x, w, out)
    out_ld = _matrix(out, "out", N, x.shape[0])
    h = _handle(dev, stream)
    B.moe_grouped_mm(dt, x, ld, w, w_e, w_n, offsets, E, x.shape[0], N, K, out, out_ld, _workspace(dev, h),
                     B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    return out


def grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Gradient of grouped_mm by x: dx[r] = w[e]^T dy[r]; dy [rows, N], w [E, N, K] -> [rows, K]."""
    dev = dy.device
    _on(dev, w=w, offsets=offsets, out=out)
    w_e, w_n = _bank(w, "w")
    E, N, K = w.shape
    ld = _matrix(dy, "dy", N)
    _check_offsets(offsets, E)
    if out is None:
        out = torch.empty((dy.shape[0], K), dtype=dy.dtype, device=dev)
    dt = _half("grouped_mm_dx", dy, w, out)
    out_ld = _matrix(out, "out", K, dy.shape[0])
    h = _handle(dev, stream)
    B.moe_grouped_mm_dx(dt, dy, ld, w, w_e, w_n, offsets, E, dy.shape[0], N, K, out, out_ld, _workspace(dev, h),
                        B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    return out


def grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm by w: dw[e] = sum over the rows of e of dy[r] x[r]^T; dy [rows, N], x [rows, K]
    -> [E, N, K], in out_dtype (the operands' type or float32).  accumulate adds to a float32 out."""
    dev = dy.device
    _on(dev, x=x, offsets=offsets, out=out)
    N, K, E = dy.shape[-1], x.shape[-1], offsets.shape[0] - 1
    ld = _matrix(dy, "dy")
    x_ld = _matrix(x, "x", None, dy.shape[0])
    _check_offsets(offsets, E)
    dt = _half("grouped_mm_dw", dy, x)
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("grouped_mm_dw: accumulate needs a float32 out")
    if out is None:
        out = torch.empty((E, N, K), dtype=out_dtype or dy.dtype, device=dev)
    if tuple(out.shape) != (E, N, K) or out.dtype not in (dy.dtype, torch.float32) or (
            out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out: {out.dtype} {tuple(out.shape)}, expected [{E}, {N}, {K}] of {out_dtype or dy.dtype}")
    o_e, o_n = _bank(out, "out")
    h = _handle(dev, stream)
    B.moe_grouped_mm_dw(dt, dy, ld, x, x_ld, offsets, E, dy.shape[0], N, K, _DTYPE[out.dtype], int(accumulate), out,
                        o_e, o_n, _workspace(dev, h), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    return out


class GroupedLinear(torch.autograd.Function):
    """grouped_mm with its gradients by x and w."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return grouped_mm(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = grouped_mm_dx(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = grouped_mm_dw(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """Differentiable grouped_mm.  Every row must belong to an expert (offsets from 0 to rows)."""
    return GroupedLinear.apply(x, w, offsets)


def quant_fp8_block(x: torch.Tensor, rows: Optional[torch.Tensor] = None, gated: bool = False,
                    out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """(q, scale): rows of x (those that the int32 index `rows` names, in its order) as E4M3 with one fp32
    scale per 128 columns; gated: of silu(x[:, :K]) * x[:, K:] with K half of x's columns.  scale has shape
    [rows, ceil(K / 128)], in any strides."""
    dev = x.device
    _on(dev, rows=rows, out=out, scale=scale)
    dt = _half("quant_fp8_block", x)
    ld = _matrix(x, "x")
    K = x.shape[1]
    if gated:
        if K % 2:
            raise ValueError(f"x: {K} columns do not split into gate and up halves")
        K //= 2
    R = x.shape[0]
    if rows is not None:
        if rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise ValueError(f"rows: expected a contiguous int32 vector, got {rows.dtype} {tuple(rows.shape)}")
        R = rows.shape[0]
    G = -(-K // BLOCK)
    if out is None:
        out = torch.empty((R, K), dtype=torch.float8_e4m3fn, device=dev)
    elif out.dtype != torch.float8_e4m3fn:
        raise ValueError(f"out: {out.dtype}, expected float8_e4m3fn")
    if scale is None:
        scale = torch.empty((R, G), dtype=torch.float32, device=dev)
    elif scale.dtype != torch.float32 or tuple(scale.shape) != (R, G):
        raise ValueError(f"scale: {scale.dtype} {tuple(scale.shape)}, expected float32 [{R}, {G}]")
    out_ld = _matrix(out, "out", K, R)
    B.moe_quant_fp8_block(dt, x, ld, x.shape[0], rows, R, K, int(gated), out, out_ld, scale,
                          (scale.stride(0), scale.stride(1)), _handle(dev, stream))
    return out, scale


def gemm_fp8_block(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                   offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Block-scaled FP8 product: x [rows, K] with x_scale [rows, ceil(K / 128)], w [N, K] with w_scale
    [ceil(N / 128), ceil(K / 128)] -> [rows, N]; with offsets, w and w_scale have a leading expert dimension
    and the rows of expert e take w[e]."""
    dev = x.device
    _on(dev, x_scale=x_scale, w=w, w_scale=w_scale, offsets=offsets, out=out)
    if offsets is None:
        w, w_scale = w.unsqueeze(0), w_scale.unsqueeze(0)
    if x.dtype != torch.float8_e4m3fn or w.dtype != torch.float8_e4m3fn:
        raise ValueError(f"gemm_fp8_block: float8_e4m3fn operands expected, got {x.dtype} and {w.dtype}")
    w_e, w_n = _bank(w, "w")
    E, N, K = w.shape
    ld = _matrix(x, "x", K)
    R, G = x.shape[0], -(-K // BLOCK)
    if x_scale.dtype != torch.float32 or tuple(x_scale.shape) != (R, G):
        raise ValueError(f"x_scale: {x_scale.dtype} {tuple(x_scale.shape)}, expected float32 [{R}, {G}]")
    if w_scale.dtype != torch.float32 or tuple(w_scale.shape) != (E, -(-N // BLOCK), G):
        raise ValueError(f"w_scale: {w_scale.dtype} {tuple(w_scale.shape)}, expected float32 "
                         f"[{E}, {-(-N // BLOCK)}, {G}]")
    if offsets is not None:
        _check_offsets(offsets, E)
    if out is None:
        out = torch.empty((R, N), dtype=out_dtype, device=dev)
    if out.dtype not in _DTYPE:
        raise ValueError(f"out: {out.dtype}, expected bfloat16, float16 or float32")
    out_ld = _matrix(out, "out", N, R)
    h = _handle(dev, stream)
    B.moe_gemm_fp8_block(x, ld, x_scale, (x_scale.stride(0), x_scale.stride(1)), w, (w_e, w_n), w_scale,
                         w_scale.stride(), offsets, E, R, N, K, _DTYPE[out.dtype], out, out_ld, _workspace(dev, h),
                         B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    return out
