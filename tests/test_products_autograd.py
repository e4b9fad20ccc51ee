"""Derivatives of grouped_linear of the first and second order: on the CPU with the
three products replaced by their formulas in 64 bits, on a GPU with small whole
numbers, for which every product and sum is exact in fp16 and fp32."""
import pytest
import torch

from weight_only_bit_moe_gb300 import products as P

SIZES, N, K = [3, 0, 4], 5, 6
ROWS = {False: 7, True: 9}  # partial: two rows of no expert


def offsets(device="cpu"):
    return torch.tensor([0, 3, 3, 7], dtype=torch.int32, device=device)


def groups(off):
    o = off.tolist()
    return enumerate(zip(o[:-1], o[1:]))


@torch.no_grad()  # like a kernel: autograd sees nothing of it
def by_row(a, w, off, out, forward):
    if out is None:
        out = a.new_empty(a.shape[0], w.shape[1 if forward else 2]).fill_(float("nan"))
    for e, (i, j) in groups(off):
        out[i:j] = a[i:j] @ (w[e].t() if forward else w[e])
    return out


@torch.no_grad()
def dw_of(dy, x, off):
    return torch.stack([dy[i:j].t() @ x[i:j] for _, (i, j) in groups(off)])


@pytest.fixture
def in_64_bits(monkeypatch):
    monkeypatch.setattr(P, "grouped_mm", lambda x, w, off, out=None: by_row(x, w, off, out, True))
    monkeypatch.setattr(P, "grouped_mm_dx", lambda dy, w, off, out=None: by_row(dy, w, off, out, False))
    monkeypatch.setattr(P, "grouped_mm_dw", dw_of)


def inputs(partial, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(ROWS[partial], K, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(len(SIZES), N, K, generator=g, dtype=torch.float64, requires_grad=True)
    return x, w


@pytest.mark.parametrize("partial", [False, True])
def test_gradients_against_differences(in_64_bits, partial):
    x, w = inputs(partial)
    assert torch.autograd.gradcheck(lambda x, w: P.grouped_linear(x, w, offsets(), partial), (x, w))


@pytest.mark.parametrize("partial", [False, True])
def test_second_derivatives_against_differences(in_64_bits, partial):
    x, w = inputs(partial)
    assert torch.autograd.gradgradcheck(lambda x, w: P.grouped_linear(x, w, offsets(), partial), (x, w))


def penalised(y, x, w):
    """A loss with the gradients of another inside: |y|^2 + |d/dx|^2 + |d/dw|^2."""
    loss = y.square().sum()
    gx, gw = torch.autograd.grad(loss, (x, w), create_graph=True)
    return loss + gx.square().sum() + gw.square().sum()


@pytest.mark.parametrize("partial", [False, True])
def test_a_loss_with_gradients_inside(in_64_bits, partial):
    x, w = inputs(partial, 1)
    got = torch.autograd.grad(penalised(P.grouped_linear(x, w, offsets(), partial), x, w), (x, w))
    parts = [x[i:j] @ w[e].t() for e, (i, j) in groups(offsets())]
    if partial:
        parts.append(x[7:] @ torch.zeros_like(w[0]).t())
    want = torch.autograd.grad(penalised(torch.cat(parts), x, w), (x, w))
    for g, r in zip(got, want):
        torch.testing.assert_close(g, r, rtol=1e-12, atol=1e-12)


def test_an_ordinary_backward_pass_records_nothing(in_64_bits):
    x, w = inputs(False, 2)
    P.grouped_linear(x, w, offsets()).sum().backward()
    assert x.grad.grad_fn is None and w.grad.grad_fn is None
    assert torch.equal(x.grad, by_row(torch.ones(7, N, dtype=torch.float64), w.detach(), offsets(), None, False))


@pytest.mark.gpu
@pytest.mark.parametrize("partial", [False, True])
def test_second_derivatives_on_gpu(partial):
    """<h, dx> + <k, dw> for the gradients dx, dw of <dy, y>: its gradients by x, w and dy are those of the
    64-bit formulas, bit for bit (entries of at most 2 in magnitude, sums of at most 64 products of three)."""
    from gpu_util import need_gpu
    need_gpu()
    off = torch.tensor([0, 19, 19, 60], dtype=torch.int32, device="cuda")
    rows, n, k = 64 if partial else 60, 24, 16
    g = torch.Generator("cuda").manual_seed(3)

    def whole(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").to(torch.float16)

    x, w, dy = whole(rows, k), whole(3, n, k), whole(rows, n)
    h, q = whole(rows, k), whole(3, n, k)
    for t in (x, w, dy):
        t.requires_grad_()
    y = P.grouped_linear(x, w, off, partial)
    dx, dw = torch.autograd.grad(y, (x, w), dy, create_graph=True)
    got = torch.autograd.grad((dx.double() * h.double()).sum() + (dw.double() * q.double()).sum(), (x, w, dy))
    x, w, dy, h, q = (t.detach().double() for t in (x, w, dy, h, q))
    end = torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
    end[:60] = 1
    zeros = lambda t, width: torch.zeros(rows, width, dtype=torch.float64, device="cuda")  # noqa: E731
    want = (by_row(dy, q, off, zeros(x, k), False), dw_of(dy, h, off),
            by_row(x, q, off, zeros(dy, n), True) + by_row(h, w, off, zeros(dy, n), True))
    for a, b in zip(got, want):
        assert torch.equal(a.double(), b)
