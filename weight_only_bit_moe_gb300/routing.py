"""PyTorch-facing calls of include/moe_routing.h: the experts of each token with their
weights, which the layer and the products take, and the balance loss that keeps the
experts evenly used while a router is trained::

    weights, ids = route(logits, top_k, score="sigmoid", bias=bias)      # differentiable by the logits
    out = layer(x, ids, weights)

    counts = expert_counts(ids, num_experts, offsets)                    # of each sequence
    loss = loss + 0.01 * balance_loss(logits, counts, offsets).mean()    # differentiable by the logits
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from . import products as P

SCORE = {"softmax": B.MOE_SCORE_SOFTMAX, "sigmoid": B.MOE_SCORE_SIGMOID}
MAX_EXPERTS = 1024


def _score(score: str) -> int:
    code = SCORE.get(score)
    if code is None:
        raise ValueError(f"score {score!r}, expected one of {sorted(SCORE)}")
    return code


def _logits(logits: torch.Tensor) -> Tuple[int, int, int, int]:
    """(type, tokens, experts, row stride)."""
    tokens, experts = P._dims(logits, "logits", 2)
    code = P._DTYPE.get(logits.dtype)
    if code is None:
        raise ValueError(f"logits of {logits.dtype}, expected bfloat16, float16 or float32")
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"logits of {experts} experts, at most {MAX_EXPERTS}")
    ld, step = logits.stride()
    if step != 1 or ld < experts:
        ld = P._rows(logits, "logits", experts, tokens)
    return code, tokens, experts, ld


def _dlogits(out: Optional[torch.Tensor], logits: torch.Tensor, stream) -> Tuple[torch.Tensor, int]:
    tokens, experts = logits.shape
    if out is None:
        return P._empty((tokens, experts), logits.dtype, logits, stream), experts
    if out.dtype is not logits.dtype:
        raise ValueError(f"out: {out.dtype}, expected {logits.dtype}")
    return out, P._rows(out, "out", experts, tokens)


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, shape) -> int:
    """Address of a contiguous tensor of that type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {list(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def topk_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
               renormalize: bool = True, scale: float = 1.0, weights: Optional[torch.Tensor] = None,
               ids: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(weights float32, ids int32), both [tokens, top_k], of logits [tokens, experts]: the top_k experts of the largest
    score plus bias (float32 [experts]), largest first, equal ones by number; their scores (softmax over the experts,
    or the sigmoid of each) as weights, divided by the chosen ones' sum if renormalize, times scale.

    Experts with logits of -inf are not chosen: id -1 and weight 0 stand in slots left over.  A token with a NaN or
    +inf gets ids -1 and weights NaN."""
    dev = P._device(logits, bias, weights, ids)
    if dev != P._current_device():
        with torch.cuda.device(dev):
            return topk_route(logits, top_k, score, bias, renormalize, scale, weights, ids, stream)
    code, tokens, experts, ld = _logits(logits)
    how = _score(score)
    if not 1 <= top_k <= min(experts, B.MOE_MAX_TOP_K):
        raise ValueError(f"top_k {top_k} of {experts} experts, at most {B.MOE_MAX_TOP_K}")
    bias_at = 0 if bias is None else _vector(bias, "bias", torch.float32, (experts,))
    if weights is None:
        weights = P._empty((tokens, top_k), torch.float32, logits, stream)
        weights_at = weights.data_ptr()
    else:
        weights_at = _vector(weights, "weights", torch.float32, (tokens, top_k))
    if ids is None:
        ids = P._empty((tokens, top_k), torch.int32, logits, stream)
        ids_at = ids.data_ptr()
    else:
        ids_at = _vector(ids, "ids", torch.int32, (tokens, top_k))
    if stream is not None:
        P._used_on(stream, logits, bias, weights, ids)
    rc = B.route(code, logits.data_ptr(), ld, bias_at, tokens, experts, top_k, how, 1 if renormalize else 0, scale,
                 weights_at, ids_at, P._handle(dev, stream))
    if rc:
        raise B.MoeError("moe_route", rc)
    return weights, ids


def topk_route_grad(dweights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                    renormalize: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Gradient of topk_route's weights by the logits, for the ids that it chose: dweights float32 [tokens, top_k] ->
    [tokens, experts] of the logits' type."""
    dev = P._device(logits, dweights, ids, out)
    if dev != P._current_device():
        with torch.cuda.device(dev):
            return topk_route_grad(dweights, logits, ids, score, renormalize, scale, out, stream)
    code, tokens, experts, ld = _logits(logits)
    how = _score(score)
    top_k = P._dims(ids, "ids", 2)[1]
    if not 1 <= top_k <= min(experts, B.MOE_MAX_TOP_K):
        raise ValueError(f"ids of {top_k} slots for {experts} experts, at most {B.MOE_MAX_TOP_K}")
    ids_at = _vector(ids, "ids", torch.int32, (tokens, top_k))
    if dweights.dtype is not torch.float32:
        raise ValueError(f"dweights: {dweights.dtype}, expected float32")
    dw_ld = P._rows(dweights, "dweights", top_k, tokens)
    out, out_ld = _dlogits(out, logits, stream)
    if stream is not None:
        P._used_on(stream, dweights, logits, ids, out)
    rc = B.route_grad(code, dweights.data_ptr(), dw_ld, logits.data_ptr(), ld, ids_at, tokens, experts, top_k,
                      how, 1 if renormalize else 0, scale, out.data_ptr(), out_ld, P._handle(dev, stream))
    if rc:
        raise B.MoeError("moe_route_grad", rc)
    return out


class Route(torch.autograd.Function):
    """topk_route with the weights' gradient by the logits."""

    @staticmethod
    def forward(ctx, logits, top_k, score, bias, renormalize, scale):
        weights, ids = topk_route(logits, top_k, score, bias, renormalize, scale)
        ctx.save_for_backward(logits, ids)
        ctx.how = score, renormalize, scale
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        return topk_route_grad(dweights.contiguous(), logits, ids, *ctx.how), None, None, None, None, None


def route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          renormalize: bool = True, scale: float = 1.0) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable topk_route: the weights have a gradient by the logits (the choice, and so the bias, has none)."""
    return Route.apply(logits, top_k, score, bias, renormalize, scale)


def _sequences(offsets: Optional[torch.Tensor]) -> Tuple[int, int]:
    """Address of the offsets and number of sequences (None: one of all tokens)."""
    if offsets is None:
        return 0, 1
    S = P._dims(offsets, "offsets", 1)[0] - 1
    if S < 1:
        raise ValueError("offsets: no sequence")
    P._check_offsets(offsets, S)
    return offsets.data_ptr(), S


def expert_counts(ids: torch.Tensor, num_experts: int, offsets: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """How often each expert stands among ids int32 [tokens, top_k]: int32 [num_experts], or with offsets int32 [S + 1]
    [S, num_experts] for the tokens offsets[s]:offsets[s + 1] of each sequence.  Other ids, such as -1, count
    nowhere."""
    dev = P._device(ids, offsets, out)
    if dev != P._current_device():
        with torch.cuda.device(dev):
            return expert_counts(ids, num_experts, offsets, out, stream)
    tokens, top_k = P._dims(ids, "ids", 2)
    if ids.dtype is not torch.int32:
        raise ValueError(f"ids: {ids.dtype}, expected int32")
    if not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError(f"{num_experts} experts, at most {MAX_EXPERTS}")
    ld = P._rows(ids, "ids", top_k, tokens)
    at, S = _sequences(offsets)
    shape = (num_experts,) if offsets is None else (S, num_experts)
    if out is None:
        out = P._empty(shape, torch.int32, ids, stream)
        out_at = out.data_ptr()
    else:
        out_at = _vector(out, "out", torch.int32, shape)
    if stream is not None:
        P._used_on(stream, ids, offsets, out)
    h = P._handle(dev, stream)
    rc = B.expert_counts(ids.data_ptr(), ld, tokens, top_k, at, S, num_experts, out_at,
                         P._workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError("moe_expert_counts", rc)
    return out


def balance(logits: torch.Tensor, counts: torch.Tensor, offsets: Optional[torch.Tensor] = None,
            score: str = "softmax", stream=None) -> torch.Tensor:
    """Balance loss, float32: E sum_e f_e p_e with f_e = counts[e] / sum of counts and p_e the mean over the tokens of
    expert e's score (softmax, or sigmoids divided by their sum); 1 for even counts.  counts int32 [E] as
    expert_counts gives them, or those of a larger batch -> a scalar; with offsets, [S, E] -> [S], one loss for the
    tokens of each sequence."""
    dev = P._device(logits, counts, offsets)
    if dev != P._current_device():
        with torch.cuda.device(dev):
            return balance(logits, counts, offsets, score, stream)
    code, tokens, experts, ld = _logits(logits)
    how = _score(score)
    at, S = _sequences(offsets)
    counts_at = _vector(counts, "counts", torch.int32, (experts,) if offsets is None else (S, experts))
    loss = P._empty(() if offsets is None else (S,), torch.float32, logits, stream)
    if stream is not None:
        P._used_on(stream, logits, counts, offsets, loss)
    h = P._handle(dev, stream)
    rc = B.balance_loss(code, logits.data_ptr(), ld, tokens, experts, counts_at, at, S, how, loss.data_ptr(),
                        P._workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError("moe_balance_loss", rc)
    return loss


def balance_grad(dloss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor,
                 offsets: Optional[torch.Tensor] = None, score: str = "softmax", out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Gradient of balance by the logits, the counts held fixed: dloss float32, a scalar or [S] -> [tokens, experts] of
    the logits' type; zeros for tokens of no sequence."""
    dev = P._device(logits, dloss, counts, offsets, out)
    if dev != P._current_device():
        with torch.cuda.device(dev):
            return balance_grad(dloss, logits, counts, offsets, score, out, stream)
    code, tokens, experts, ld = _logits(logits)
    how = _score(score)
    at, S = _sequences(offsets)
    counts_at = _vector(counts, "counts", torch.int32, (experts,) if offsets is None else (S, experts))
    dloss_at = _vector(dloss, "dloss", torch.float32, () if offsets is None else (S,))
    out, out_ld = _dlogits(out, logits, stream)
    if stream is not None:
        P._used_on(stream, dloss, logits, counts, offsets, out)
    h = P._handle(dev, stream)
    rc = B.balance_loss_grad(code, dloss_at, logits.data_ptr(), ld, tokens, experts, counts_at, at, S, how,
                             out.data_ptr(), out_ld, P._workspace(dev, h, stream), B.MOE_PRODUCTS_WORKSPACE_BYTES, h)
    if rc:
        raise B.MoeError("moe_balance_loss_grad", rc)
    return out


class BalanceLoss(torch.autograd.Function):
    """balance with its gradient by the logits."""

    @staticmethod
    def forward(ctx, logits, counts, offsets, score):
        ctx.save_for_backward(logits, counts, offsets)
        ctx.score = score
        return balance(logits, counts, offsets, score)

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        logits, counts, offsets = ctx.saved_tensors
        return balance_grad(dloss.contiguous(), logits, counts, offsets, ctx.score), None, None, None


def balance_loss(logits: torch.Tensor, counts: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                 score: str = "softmax") -> torch.Tensor:
    """Differentiable balance (by the logits; the counts are constants)."""
    return BalanceLoss.apply(logits, counts, offsets, score)
