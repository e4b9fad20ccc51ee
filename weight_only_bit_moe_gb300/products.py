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

import threading
from typing import Optional, Tuple

import torch

from . import binding as B

BLOCK = 128  # columns per FP8 scale; also rows of a weight block
_HALF = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16}
_DTYPE = {torch.bfloat16: B.MOE_BF16, torch.float16: B.MOE_FP16, torch.float32: B.MOE_FP32}

# One workspace per device and stream, as the kernels of one stream run one after another: (address, tensor).
_workspaces = {}
# Those of captured calls, by device, stream and capture: (address, tensor, word that tells whether the graph is gone).
_captured = {}
_workspace_lock = threading.Lock()


def _handle(device: int, stream) -> int:
    """CUDA handle of the stream (default: the device's current one)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _workspace(device: int, handle: int, stream=None) -> int:
    """Address of the workspace of this device and stream (`stream` as the caller gave it).  A captured call never
    takes it: the graph may be replayed on any stream, beside calls on this one."""
    if torch._C._cuda_isCurrentStreamCapturing() if stream is None else B.moe_capture_id(handle):
        return _captured_workspace(device, handle)
    ws = _workspaces.get((device, handle))
    return ws[0] if ws is not None else _new_workspace(device, handle)


def _new_workspace(device: int, handle: int) -> int:
    with _workspace_lock:
        if (device, handle) not in _workspaces:
            ws = _zeroed(device)
            _workspaces[(device, handle)] = (ws.data_ptr(), ws)
        return _workspaces[(device, handle)][0]


def _captured_workspace(device: int, handle: int) -> int:
    """Address of the workspace of the capture that the stream is in, on that stream: branches of a graph may run
    at one time.  It is kept until the graph is gone, and then serves another capture."""
    key = (device, handle, B.moe_capture_id(handle))
    ws = _captured.get(key)
    if ws is None:
        with _workspace_lock:
            ended = next((k for k, (_, _, gone) in _captured.items() if k[0] == device and gone.contents.value), None)
            ws = _zeroed(device, None if ended is None else _captured.pop(ended)[1])
            ws = _captured[key] = (ws.data_ptr(), ws, B.moe_capture_watch(handle))
    return ws[0]


def _zeroed(device: int, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A workspace (a new one unless given) whose head is zeros when this returns; one that is given keeps its
    status, which nobody may have read.  Also while the thread captures: the kernels leave their counters at zero,
    so a graph needs no fill of its own, and memory that is not the graph's is not shared with its other nodes."""
    mode = B.moe_capture_mode(2)  # relaxed
    try:
        side = torch.cuda.Stream(device)
        while B.moe_capture_id(side):  # (streams are handed out in turn)
            side = torch.cuda.Stream(device)
        with torch.cuda.stream(side):
            first = 4  # past the status word
            if ws is None:
                ws = torch.empty(B.MOE_PRODUCTS_WORKSPACE_BYTES, dtype=torch.uint8, device=torch.device("cuda", device))
                first = 0
            ws[first:B.MOE_PRODUCTS_WORKSPACE_HEAD_BYTES].zero_()
        side.synchronize()
    finally:
        B.moe_capture_mode(mode)
    return ws


def _empty(shape, dtype: torch.dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """An output on `like`'s device of a kernel that runs on `stream`, from that stream's memory."""
    device = like.device  # (a device object: torch takes 2 us longer to make a tensor for a device number)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _used_on(stream, *tensors: Optional[torch.Tensor]) -> None:
    """Tells the allocator that a kernel on `stream` uses these tensors: their memory is not given out again
    before it has run."""
    for t in tensors:
        if t is not None:
            t.record_stream(torch.cuda.ExternalStream(stream, device=t.device) if isinstance(stream, int) else stream)


def products_status(device="cuda", stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status of its products and of those in the
    device's graphs, whose replays it waits for on every stream: MOE_OK, MOE_ERR_TIMEOUT or MOE_ERR_INVALID
    (offsets that decrease or leave the rows)."""
    index = torch.device(device).index
    index = torch.cuda.current_device() if index is None else index
    if index != _current_device():
        with torch.cuda.device(index):
            return products_status(torch.device("cuda", index), stream)
    handle = _handle(index, stream)
    status = [B.moe_get_status(_workspace(index, handle), handle)]
    graphs = [ws for key, (ws, _, _) in list(_captured.items()) if key[0] == index]
    if graphs:
        torch.cuda.synchronize(index)
        status += [B.moe_get_status(ws, handle) for ws in graphs]
    return next((s for s in (B.MOE_ERR_CUDA, B.MOE_ERR_TIMEOUT) if s in status),
                next((s for s in status if s != B.MOE_OK), B.MOE_OK))


# The checks below read each attribute of a tensor once: for a decode step they are most of a call's host time.

def _rows(t: torch.Tensor, name: str, width: int, rows: int) -> int:
    """Row stride of a row-major matrix of that shape."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != width:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [{rows}, {width}]")
    s0, s1 = t.stride()
    if s1 != 1 and width > 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous (strides {t.stride()})")
    if s0 < width:
        if rows > 1:
            raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
        return width
    return s0


def _bank(t: torch.Tensor, name: str, shape) -> Tuple[int, int]:
    """(expert, row) strides of a bank [E, N, K]."""
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous (strides {t.stride()})")
    if s1 < shape[2]:
        if shape[1] > 1:
            raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
        return s0, shape[2]
    return s0, s1


def _dims(t: torch.Tensor, name: str, dims: int):
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {dims} dimensions")
    return shape


def _device(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """Index of the GPU that holds every tensor (tensors that are None are skipped)."""
    device = first.get_device()
    if device < 0:
        raise ValueError(f"the products run on a GPU, not on {first.device}")
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors on {first.device} and {t.device}")
    return device


def _current_device() -> int:
    """The calling thread's device.  The library launches there, so a call with operands on another GPU starts
    again with that one current."""
    return torch._C._cuda_getDevice()


def _check_offsets(offsets: torch.Tensor, E: int) -> None:
    if offsets.dtype is not torch.int32 or offsets.numel() != E + 1 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError(f"offsets: expected contiguous int32 [{E + 1}], got {offsets.dtype} {tuple(offsets.shape)}")


def _types(name: str, *tensors: torch.Tensor) -> ValueError:
    return ValueError(f"{name}: operands of one type, bfloat16 or float16, expected; got "
                      f"{', '.join(str(t.dtype) for t in tensors)}")


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


def _by_row(fn: str, name: str, a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
            out: Optional[torch.Tensor], stream, forward: bool) -> torch.Tensor:
    dev = _device(a, w, offsets, out)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _by_row(fn, name, a, w, offsets, out, stream, forward)
    rows, a_width = _dims(a, name, 2)
    E, N, K = shape = _dims(w, "w", 3)
    width, out_width = (K, N) if forward else (N, K)
    dtype = a.dtype
    code = _HALF.get(dtype)
    if code is None or w.dtype is not dtype:
        raise _types(fn, a, w)
    w_e, w_n, step = w.stride()
    if step != 1 or w_n < K:
        w_e, w_n = _bank(w, "w", shape)
    ld, step = a.stride()
    if a_width != width or step != 1 or ld < width:
        ld = _rows(a, name, width, rows)
    _check_offsets(offsets, E)
    if out is None:
        out = _empty((rows, out_width), dtype, a, stream)
        out_ld = out_width
    else:
        if out.dtype is not dtype:
            raise _types(fn, a, out)
        out_ld = _rows(out, "out", out_width, rows)
    if stream is not None:
        _used_on(stream, a, w, offsets, out)
    h = _handle(dev, stream)
    rc = B.function(fn)(code, a.data_ptr(), ld, w.data_ptr(), w_e, w_n, offsets.data_ptr(), E, rows, N, K,
                        out.data_ptr(), out_ld, _workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError(fn, rc)
    return out


def grouped_mm(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows r of expert e: x [rows, K], w [E, N, K] -> [rows, N]."""
    return _by_row("moe_grouped_mm", "x", x, w, offsets, out, stream, True)


def grouped_mm_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Gradient of grouped_mm by x: dx[r] = w[e]^T dy[r]; dy [rows, N], w [E, N, K] -> [rows, K]."""
    return _by_row("moe_grouped_mm_dx", "dy", dy, w, offsets, out, stream, False)


def grouped_mm_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient of grouped_mm by w: dw[e] = sum over the rows of e of dy[r] x[r]^T; dy [rows, N], x [rows, K]
    -> [E, N, K], in out_dtype (the operands' type or float32).  accumulate adds to a float32 out."""
    dev = _device(dy, x, offsets, out)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return grouped_mm_dw(dy, x, offsets, out, out_dtype, accumulate, stream)
    rows, N = _dims(dy, "dy", 2)
    K = _dims(x, "x", 2)[1]
    E = _dims(offsets, "offsets", 1)[0] - 1
    ld = _rows(dy, "dy", N, rows)
    x_ld = _rows(x, "x", K, rows)
    _check_offsets(offsets, E)
    dtype = dy.dtype
    code = _HALF.get(dtype)
    if code is None or x.dtype is not dtype:
        raise _types("grouped_mm_dw", dy, x)
    if out_dtype is None:
        out_dtype = dtype if out is None else out.dtype
    if out_dtype is not dtype and out_dtype is not torch.float32:
        raise ValueError(f"grouped_mm_dw: {out_dtype} gradients, expected {dtype} or float32")
    if accumulate and (out is None or out_dtype is not torch.float32):
        raise ValueError("grouped_mm_dw: accumulate needs a float32 out")
    if out is None:
        out = _empty((E, N, K), out_dtype, dy, stream)
        o_e, o_n = N * K, K
    else:
        if tuple(out.shape) != (E, N, K) or out.dtype is not out_dtype:
            raise ValueError(f"out: {out.dtype} {tuple(out.shape)}, expected {out_dtype} [{E}, {N}, {K}]")
        o_e, o_n = _bank(out, "out", out.shape)
    if stream is not None:
        _used_on(stream, dy, x, offsets, out)
    h = _handle(dev, stream)
    rc = B.function("moe_grouped_mm_dw")(
        code, dy.data_ptr(), ld, x.data_ptr(), x_ld, offsets.data_ptr(), E, rows, N, K,
        code if out_dtype is dtype else B.MOE_FP32, 1 if accumulate else 0, out.data_ptr(), o_e, o_n,
        _workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError("moe_grouped_mm_dw", rc)
    return out


# y = grouped_mm(x, w), dx = grouped_mm_dx(dy, w) and dw = grouped_mm_dw(dy, x) are bilinear, and the gradients of each
# are the other two, so the three have derivatives of any order.  In an ordinary backward pass autograd records
# nothing, and the kernels are called without its bookkeeping.

def _by_row_zeroed(fn, a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, partial: bool, width: int):
    return fn(a, w, offsets, out=a.new_zeros((a.shape[0], width)) if partial else None)


def _mm(x, w, offsets, partial):
    if torch.is_grad_enabled():
        return GroupedLinear.apply(x, w, offsets, partial)
    return _by_row_zeroed(grouped_mm, x, w, offsets, partial, w.shape[1])


def _mm_dx(dy, w, offsets, partial):
    if torch.is_grad_enabled():
        return GroupedLinearDx.apply(dy, w, offsets, partial)
    return _by_row_zeroed(grouped_mm_dx, dy, w, offsets, partial, w.shape[2])


def _mm_dw(dy, x, offsets, partial):
    return GroupedLinearDw.apply(dy, x, offsets, partial) if torch.is_grad_enabled() else grouped_mm_dw(dy, x, offsets)


class GroupedLinear(torch.autograd.Function):
    """grouped_mm with its gradients by x and w."""

    @staticmethod
    def forward(ctx, x, w, offsets, partial):
        ctx.save_for_backward(x, w, offsets)
        ctx.partial = partial
        return _by_row_zeroed(grouped_mm, x, w, offsets, partial, w.shape[1])

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = _mm_dx(dy, w, offsets, ctx.partial) if ctx.needs_input_grad[0] else None
        dw = _mm_dw(dy, x, offsets, ctx.partial) if ctx.needs_input_grad[1] else None
        return dx, dw, None, None


class GroupedLinearDx(torch.autograd.Function):
    """grouped_mm_dx with its gradients by dy and w."""

    @staticmethod
    def forward(ctx, dy, w, offsets, partial):
        ctx.save_for_backward(dy, w, offsets)
        ctx.partial = partial
        return _by_row_zeroed(grouped_mm_dx, dy, w, offsets, partial, w.shape[2])

    @staticmethod
    def backward(ctx, g):
        dy, w, offsets = ctx.saved_tensors
        g = g.contiguous()
        d_dy = _mm(g, w, offsets, ctx.partial) if ctx.needs_input_grad[0] else None
        d_w = _mm_dw(dy, g, offsets, ctx.partial) if ctx.needs_input_grad[1] else None
        return d_dy, d_w, None, None


class GroupedLinearDw(torch.autograd.Function):
    """grouped_mm_dw with its gradients by dy and x."""

    @staticmethod
    def forward(ctx, dy, x, offsets, partial):
        ctx.save_for_backward(dy, x, offsets)
        ctx.partial = partial
        return grouped_mm_dw(dy, x, offsets)

    @staticmethod
    def backward(ctx, g):
        dy, x, offsets = ctx.saved_tensors
        g = g.contiguous()
        d_dy = _mm(x, g, offsets, ctx.partial) if ctx.needs_input_grad[0] else None
        d_x = _mm_dx(dy, g, offsets, ctx.partial) if ctx.needs_input_grad[1] else None
        return d_dy, d_x, None, None


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, partial: bool = False) -> torch.Tensor:
    """Differentiable grouped_mm, its derivatives too.  Every row must belong to an expert (offsets from 0 to rows),
    unless `partial`: then the other rows, as of experts held elsewhere, give zeros and get zeros as their gradient.
    (The calls that take `out` are the kernels alone: what they return has no gradient.)"""
    return GroupedLinear.apply(x, w, offsets, partial)


def quant_fp8_block(x: torch.Tensor, rows: Optional[torch.Tensor] = None, gated: bool = False,
                    out: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """(q, scale): rows of x (those that the int32 index `rows` names, in its order) as E4M3 with one fp32
    scale per 128 columns; gated: of silu(x[:, :K]) * x[:, K:] with K half of x's columns.  scale has shape
    [rows, ceil(K / 128)], in any strides."""
    dev = _device(x, rows, out, scale)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return quant_fp8_block(x, rows, gated, out, scale, stream)
    code = _HALF.get(x.dtype)
    if code is None:
        raise _types("quant_fp8_block", x)
    x_rows, K = _dims(x, "x", 2)
    ld = _rows(x, "x", K, x_rows)
    if gated:
        if K % 2:
            raise ValueError(f"x: {K} columns do not split into gate and up halves")
        K //= 2
    R, index = x_rows, None
    if rows is not None:
        if rows.dtype is not torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise ValueError(f"rows: expected a contiguous int32 vector, got {rows.dtype} {tuple(rows.shape)}")
        R, index = rows.shape[0], rows.data_ptr()
    G = -(-K // BLOCK)
    if out is None:
        out = _empty((R, K), torch.float8_e4m3fn, x, stream)
        out_ld = K
    else:
        if out.dtype is not torch.float8_e4m3fn:
            raise ValueError(f"out: {out.dtype}, expected float8_e4m3fn")
        out_ld = _rows(out, "out", K, R)
    if scale is None:
        scale = _empty((R, G), torch.float32, x, stream)
        s_m, s_g = G, 1
    else:
        if scale.dtype is not torch.float32 or tuple(scale.shape) != (R, G):
            raise ValueError(f"scale: {scale.dtype} {tuple(scale.shape)}, expected float32 [{R}, {G}]")
        s_m, s_g = scale.stride()
    if stream is not None:
        _used_on(stream, x, rows, out, scale)
    rc = B.function("moe_quant_fp8_block")(
        code, x.data_ptr(), ld, x_rows, index, R, K, 1 if gated else 0, out.data_ptr(), out_ld, scale.data_ptr(), s_m,
        s_g, _handle(dev, stream))
    if rc:
        raise B.MoeError("moe_quant_fp8_block", rc)
    return out, scale


def gemm_fp8_block(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                   offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Block-scaled FP8 product: x [rows, K] with x_scale [rows, ceil(K / 128)], w [N, K] with w_scale
    [ceil(N / 128), ceil(K / 128)] -> [rows, N] in out_dtype (bfloat16, float16 or float32; bfloat16 unless
    out is given); with offsets, w and w_scale have a leading expert dimension and the rows of expert e take
    w[e].  Scales may have any strides."""
    dev = _device(x, x_scale, w, w_scale, offsets, out)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return gemm_fp8_block(x, x_scale, w, w_scale, offsets, out, out_dtype, stream)
    if x.dtype is not torch.float8_e4m3fn or w.dtype is not torch.float8_e4m3fn:
        raise ValueError(f"gemm_fp8_block: float8_e4m3fn operands expected, got {x.dtype} and {w.dtype}")
    if x_scale.dtype is not torch.float32 or w_scale.dtype is not torch.float32:
        raise ValueError(f"gemm_fp8_block: float32 scales expected, got {x_scale.dtype} and {w_scale.dtype}")
    if offsets is None:
        N, K = _dims(w, "w", 2)
        E, w_e, w_n = 1, 0, _rows(w, "w", K, N)
        at = None
    else:
        shape = _dims(w, "w", 3)
        E, N, K = shape
        w_e, w_n = _bank(w, "w", shape)
        _check_offsets(offsets, E)
        at = offsets.data_ptr()
    R, G, GN = _dims(x, "x", 2)[0], -(-K // BLOCK), -(-N // BLOCK)
    ld = _rows(x, "x", K, R)
    if x_scale.shape != (R, G):
        raise ValueError(f"x_scale: {tuple(x_scale.shape)}, expected [{R}, {G}]")
    if w_scale.shape != ((GN, G) if offsets is None else (E, GN, G)):
        raise ValueError(f"w_scale: {tuple(w_scale.shape)}, expected [{'' if offsets is None else f'{E}, '}{GN}, {G}]")
    ws = w_scale.stride()
    if out is None:
        out_dtype = out_dtype or torch.bfloat16
        code = _DTYPE.get(out_dtype)
    else:
        code = _DTYPE.get(out.dtype) if out_dtype is None or out_dtype is out.dtype else None
    if code is None:
        raise ValueError(f"gemm_fp8_block: out of {out_dtype if out is None else out.dtype}, expected bfloat16, "
                         "float16 or float32 and, with out_dtype, that type")
    if out is None:
        out = _empty((R, N), out_dtype, x, stream)
        out_ld = N
    else:
        out_ld = _rows(out, "out", N, R)
    s_m, s_g = x_scale.stride()
    if stream is not None:
        _used_on(stream, x, x_scale, w, w_scale, offsets, out)
    h = _handle(dev, stream)
    rc = B.function("moe_gemm_fp8_block")(
        x.data_ptr(), ld, x_scale.data_ptr(), s_m, s_g, w.data_ptr(), w_e, w_n, w_scale.data_ptr(),
        0 if offsets is None else ws[0], ws[-2], ws[-1], at, E, R, N, K, code, out.data_ptr(), out_ld,
        _workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError("moe_gemm_fp8_block", rc)
    return out
