"""References in 64 bits and error bounds for the products of include/moe_products.h.

Bounds.  A sum of T products a*b in fp32, in any order and with every addition
rounded or cut to 24 bits, is off by at most (T + 8) 2^-23 sum |a b| (the 8 covers
the products' own rounding and the joining of partial sums); rounding the result
to the output type adds half a unit in its last place, for p significant bits at
most 2^-p |y|: 2^-8 |y| for bf16, 2^-11 |y| for fp16 (2^-25 below its normal range),
2^-24 |y| for fp32."""
import torch

# a unit in the last place: relative to the value (at most), and in the subnormal range
ULP = {torch.bfloat16: (2.0 ** -7, 2.0 ** -133), torch.float16: (2.0 ** -10, 2.0 ** -24),
       torch.float32: (2.0 ** -23, 2.0 ** -149)}


def spans(offsets):
    o = offsets.tolist()
    return list(zip(o[:-1], o[1:]))


def offsets_of(sizes, first=0, device="cuda"):
    o = [first]
    for s in sizes:
        o.append(o[-1] + s)
    return torch.tensor(o, dtype=torch.int32, device=device)


def assert_within(got, ref, mag, terms, what=""):
    """|got - ref| <= the bound above, ref and mag = sum |a b| in 64 bits."""
    assert got.shape == ref.shape, (got.shape, ref.shape)
    if ref.numel() == 0:
        return
    rel, floor = ULP[got.dtype]
    bound = (terms + 8) * 2.0 ** -23 * mag + 0.5 * (rel * ref.abs() * (1 + 2.0 ** -7) + floor)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = err > bound
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} outside the bound, first {at}: "
                             f"got {float(got[at])} ref {float(ref[at])} bound {float(bound[at]):.3g}")


def ref_fwd(x, w, offsets):
    """[(rows, y, sum |x w|)] per expert."""
    out = []
    for e, (a, b) in enumerate(spans(offsets)):
        xe, we = x[a:b].double(), w[e].double()
        out.append(((a, b), xe @ we.t(), xe.abs() @ we.abs().t()))
    return out


def ref_dx(dy, w, offsets):
    out = []
    for e, (a, b) in enumerate(spans(offsets)):
        de, we = dy[a:b].double(), w[e].double()
        out.append(((a, b), de @ we, de.abs() @ we.abs()))
    return out


def ref_dw(dy, x, offsets):
    out = []
    for a, b in spans(offsets):
        de, xe = dy[a:b].double(), x[a:b].double()
        out.append((b - a, de.t() @ xe, de.abs().t() @ xe.abs()))
    return out


def spread_rows(scale, width):
    """[rows, blocks] -> [rows, width]."""
    return scale.repeat_interleave(128, 1)[:, :width]


def dequant_bank(w, ws):
    E, N, K = w.shape
    return w.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K]


def strided(t, pad, fill):
    """A copy of the matrix or bank t whose rows lie pad elements further apart, the gaps holding fill."""
    shape = list(t.shape)
    shape[-1] += pad
    # 8-bit floats are filled through their bytes
    if t.dtype == torch.float8_e4m3fn:
        base = torch.full(shape, 0x7F, dtype=torch.uint8, device=t.device).view(torch.float8_e4m3fn)
    else:
        base = torch.full(shape, fill, dtype=t.dtype, device=t.device)
    view = base[..., :t.shape[-1]]
    view.copy_(t)
    return view
