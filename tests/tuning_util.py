"""References in 64 bits and error bounds for the routing and the adapters.

Adapters (include/moe_adapters.h).  mid is a sum of T products in fp32, off by at most
(T + 8) 2^-23 sum |f x| (products_util).  It enters the second product, of R terms, with
16 significant bits at least (2^-16 |mid|, relative), so with D the bound of mid
  |out - ref| <= |scale| sum_j |s_j| (D_j + 2^-16 |mid_j|) + (R + 8) 2^-23 |scale| sum |s mid|
                 + 2^-22 |base| + half a unit of the result.
The gradients sum n products of mid, as given, and 16-bit rows:
  |grad - ref| <= |scale| (2^-16 + (n + 8) 2^-23) sum |mid in| + half a unit,
and with fp16 rows mid may be held as a pair of fp16 numbers on the scale of the
adapter's largest: 2^-36 max |mid| sum |in| more.

Routing (include/moe_routing.h).  An exponential of a difference d of logits is off by
2^-24 |d| (the difference's rounding) + 2^-22 (its own, two units) relative; a sum of E
positive ones adds E 2^-24, the quotient 2^-22: with d <= the token's range,
  rel = 2^-23 (E / 2 + range / 2 + 16)."""
import torch

from products_util import ULP


def half_unit(ref, dtype):
    rel, floor = ULP[dtype]
    return 0.5 * (rel * ref.abs() * (1 + 2.0 ** -7) + floor)


def assert_bound(got, ref, bound, what=""):
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if ref.numel() == 0:
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bound = bound + half_unit(ref, got.dtype)
    err = (got.double() - ref).abs()
    bad = err > bound
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} outside the bound, first {at}: "
                             f"got {float(got[at])} ref {float(ref[at])} bound {float(bound[at]):.3g}")


def positions(offsets, order, l):
    a, b = int(offsets[l]), int(offsets[l + 1])
    index = torch.arange(a, b, device=offsets.device)
    return index, (index if order is None else order[a:b].long())


def check_adapter(got, mid, rows_in, first, second, offsets, order, scale, base, what=""):
    """got, mid of adapter_mm (first = a, second = b) or adapter_mm_dx (first = b^T, second = a^T), as [L, R, P] and
    [L, Q, R]."""
    L, R, P = first.shape
    rows, Q = got.shape
    ref = torch.zeros(rows, Q, dtype=torch.float64, device=got.device) if base is None else base.double()
    bound = 2.0 ** -22 * ref.abs()
    for l in range(L):
        at, row = positions(offsets, order, l)
        if len(at) == 0:
            continue
        x, f, s = rows_in[row].double(), first[l].double(), second[l].double()
        c = 1.0 if scale is None else scale[l].double()
        t, mag = x @ f.t(), x.abs() @ f.abs().t()
        d = (P + 8) * 2.0 ** -23 * mag
        if mid is not None:
            assert_bound(mid[at], t, d, f"{what} mid of {l}")
        ref[row] += c * (t @ s.t())
        bound[row] += abs(c) * ((d + (2.0 ** -16 + (R + 8) * 2.0 ** -23) * t.abs()) @ s.abs().t())
    assert_bound(got, ref, bound, what)


def check_adapter_grads(da, db, dy, x, mid_x, mid_dy, offsets, order, scale, start=(None, None), what=""):
    for name, got, rows_in, mid, first in (("da", da, x, mid_dy, start[0]), ("db", db, dy, mid_x, start[1])):
        if got is None:
            continue
        fp16 = rows_in.dtype is torch.float16
        for l in range(got.shape[0]):
            at, row = positions(offsets, order, l)
            m, v = mid[at].double(), rows_in[row].double()
            c = 1.0 if scale is None else scale[l].double()
            ref, mag = c * (m.t() @ v), abs(c) * (m.abs().t() @ v.abs())
            bound = (2.0 ** -16 + (len(at) + 8) * 2.0 ** -23) * mag
            if fp16 and len(at):
                bound = bound + abs(c) * 2.0 ** -36 * m.abs().max() * v.abs().sum(0)[None]
            if name == "db":
                ref, bound = ref.t(), bound.t()
            if first is not None:
                ref = ref + first[l].double()
                bound = bound + 2.0 ** -23 * first[l].double().abs()
            assert_bound(got[l], ref, bound, f"{what} {name} of {l}")


# ---------------------------------------------------------------- routing
def ref_scores(logits, score):
    l = logits.double()
    return torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)


def ref_route(logits, top_k, score, bias, renormalize, scale):
    """(weights, ids) in 64 bits; a token's logits finite or -inf."""
    l = logits.double()
    p = ref_scores(logits, score).nan_to_num(0.0)
    keys = l.clone() if bias is None else torch.where(l == -float("inf"), l, p + bias.double())
    order = torch.sort(keys, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :top_k] == -float("inf"), -1, order.indices[:, :top_k])
    if renormalize:
        chosen = l.gather(1, ids.clamp_min(0))
        if score == "sigmoid":
            chosen = torch.nn.functional.logsigmoid(chosen)
        w = torch.softmax(torch.where(ids < 0, -float("inf"), chosen), 1).nan_to_num(0.0)
    else:
        w = torch.where(ids < 0, 0.0, p.gather(1, ids.clamp_min(0)))
    return scale * w, ids.to(torch.int32)


def rel_bound(logits):
    l = logits.double()
    low = torch.where(l == -float("inf"), float("inf"), l).amin(1)
    spread = (l.amax(1) - low).clamp_min(0.0).nan_to_num(0.0, 0.0, 0.0)
    return (2.0 ** -23 * (logits.shape[1] / 2 + spread / 2 + 16))[:, None]


def ref_route_grad(dweights, logits, ids, score, renormalize, scale):
    """(gradient, sum of the magnitudes that it is made of), by autograd of the definition in 64 bits."""
    def grad(g):
        l = logits.double().requires_grad_()
        held = (ids >= 0) & (ids < logits.shape[1])
        at = torch.where(held, ids, 0).long()
        chosen = l.gather(1, at)
        if renormalize:
            v = chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen)
            v = torch.where(held, v, torch.full_like(v, -1e300))
            w = torch.softmax(v, 1)
        else:
            w = (torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)).gather(1, at)
        w = scale * torch.where(held, w, torch.zeros_like(w))
        return torch.autograd.grad((w * g).sum(), l)[0], w.detach()

    g = dweights.double()
    ref, w = grad(g)
    p = ref_scores(logits, score)
    total = (w.abs() * g.abs()).sum(1, keepdim=True)
    mag = torch.zeros_like(ref).scatter_add_(1, ids.clamp(0, logits.shape[1] - 1).long(), w.abs() * (g.abs() + total / max(abs(scale), 1e-30)))
    if score == "softmax" and not renormalize:
        mag = mag + p * total
    return ref, mag


def ref_balance(logits, counts, offsets, score):
    """(losses, per-token gradient for dloss = 1, magnitude of that) in 64 bits."""
    l = logits.double()
    E = l.shape[1]
    p = torch.softmax(l if score == "softmax" else torch.nn.functional.logsigmoid(l), 1).nan_to_num(0.0)
    slope = p if score == "softmax" else p * torch.sigmoid(-l)
    losses, grad, mag = [], torch.zeros_like(l), torch.zeros_like(l)
    for s in range(len(offsets) - 1):
        a, b = int(offsets[s]), int(offsets[s + 1])
        c = counts[s].double()
        n = float(c.sum()) * (b - a)
        if n == 0:
            losses.append(l.new_zeros(()))
            continue
        inner = (p[a:b] * c).sum(1, keepdim=True)
        losses.append(E / n * inner.sum())
        grad[a:b] = E / n * slope[a:b] * (c - inner)
        mag[a:b] = E / n * slope[a:b] * (c + inner)
    return torch.stack(losses), grad, mag
