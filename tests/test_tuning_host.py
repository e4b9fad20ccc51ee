"""Refusals of the routing and the adapters (include/moe_routing.h, moe_adapters.h) that
need no GPU: the C entries before they touch the device, the PyTorch calls before they
call them."""
import pytest
import torch

BUF = 1 << 20  # an address on a 256-byte boundary; nothing reads it


@pytest.fixture(scope="module")
def lib():
    from weight_only_bit_moe_gb300 import build, binding
    build.build()
    return binding


def call(lib, fn, args, kw):
    args = dict(args)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return getattr(lib.load(), fn)(*args.values())


ROUTE = dict(dtype=2, logits=BUF, ld=64, bias=0, tokens=10, experts=64, top_k=4, score=0, renormalize=1, scale=1.0,
             weights=BUF, ids=BUF, stream=0)
ROUTE_GRAD = dict(dtype=2, dweights=BUF, dw_ld=4, logits=BUF, ld=64, ids=BUF, tokens=10, experts=64, top_k=4, score=0,
                  renormalize=1, scale=1.0, out=BUF, out_ld=64, stream=0)
SHARED = [dict(tokens=2 ** 31 - 65536), dict(dtype=3), dict(dtype=-1), dict(ld=63), dict(tokens=-1), dict(experts=0), dict(experts=1025, ld=1025),
          dict(top_k=0), dict(top_k=33), dict(top_k=5, experts=4), dict(score=2), dict(score=-1), dict(renormalize=2),
          dict(logits=0), dict(logits=BUF + 2), dict(ids=0), dict(ids=BUF + 2)]


@pytest.mark.parametrize("bad", SHARED + [dict(weights=0), dict(weights=BUF + 1), dict(bias=BUF + 2)], ids=str)
def test_route_refusals(lib, bad):
    assert call(lib, "moe_route", ROUTE, bad) == lib.MOE_ERR_INVALID


@pytest.mark.parametrize("bad", SHARED + [dict(dweights=0), dict(dw_ld=3), dict(out=0), dict(out_ld=63),
                                          dict(out=BUF + 2), dict(dweights=BUF + 2)], ids=str)
def test_route_grad_refusals(lib, bad):
    assert call(lib, "moe_route_grad", ROUTE_GRAD, bad) == lib.MOE_ERR_INVALID


def test_route_of_no_tokens(lib):
    assert call(lib, "moe_route", ROUTE, dict(tokens=0, logits=0, weights=0, ids=0)) == lib.MOE_OK
    assert call(lib, "moe_route_grad", ROUTE_GRAD, dict(tokens=0, logits=0, dweights=0, ids=0, out=0)) == lib.MOE_OK


def workspace(lib):
    return dict(workspace=BUF, workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES, stream=0)


COUNTS = dict(ids=BUF, ld=4, tokens=10, top_k=4, offsets=BUF, sequences=2, experts=64, counts=BUF)


@pytest.mark.parametrize("bad", [
    dict(ids=0), dict(ids=BUF + 1), dict(ld=3), dict(tokens=-1), dict(top_k=0), dict(tokens=2 ** 30, top_k=4),
    dict(tokens=2 ** 31 - 65536, top_k=1), dict(offsets=0), dict(offsets=BUF + 1), dict(sequences=0), dict(sequences=(1 << 20) + 1), dict(experts=0),
    dict(experts=1025), dict(counts=0), dict(counts=BUF + 2), dict(workspace=0), dict(workspace=BUF + 8)], ids=str)
def test_counts_refusals(lib, bad):
    assert call(lib, "moe_expert_counts", {**COUNTS, **workspace(lib)}, bad) == lib.MOE_ERR_INVALID


LOSS = dict(dtype=2, logits=BUF, ld=64, tokens=10, experts=64, counts=BUF, offsets=BUF, sequences=2, score=0, loss=BUF)
LOSS_GRAD = dict(dtype=2, dloss=BUF, logits=BUF, ld=64, tokens=10, experts=64, counts=BUF, offsets=BUF, sequences=2,
                 score=0, out=BUF, out_ld=64)
LOSS_BAD = [dict(dtype=3), dict(logits=0), dict(logits=BUF + 1), dict(ld=63), dict(tokens=-1), dict(experts=0),
            dict(experts=1025, ld=1025), dict(counts=0), dict(counts=BUF + 2), dict(offsets=0), dict(offsets=BUF + 2),
            dict(sequences=0), dict(sequences=(1 << 20) + 1), dict(score=2), dict(workspace=0), dict(workspace=BUF + 64)]


@pytest.mark.parametrize("bad", LOSS_BAD + [dict(loss=0), dict(loss=BUF + 1)], ids=str)
def test_balance_refusals(lib, bad):
    assert call(lib, "moe_balance_loss", {**LOSS, **workspace(lib)}, bad) == lib.MOE_ERR_INVALID


@pytest.mark.parametrize("bad", LOSS_BAD + [dict(dloss=0), dict(dloss=BUF + 1), dict(out=0), dict(out_ld=63),
                                            dict(out=BUF + 2)], ids=str)
def test_balance_grad_refusals(lib, bad):
    assert call(lib, "moe_balance_loss_grad", {**LOSS_GRAD, **workspace(lib)}, bad) == lib.MOE_ERR_INVALID


def test_small_workspaces(lib):
    small = dict(workspace=BUF, workspace_bytes=lib.MOE_PRODUCTS_WORKSPACE_BYTES - 1, stream=0)
    for fn, args in (("moe_expert_counts", COUNTS), ("moe_balance_loss", LOSS), ("moe_balance_loss_grad", LOSS_GRAD),
                     ("moe_adapter_mm", MM), ("moe_adapter_mm_dx", MM), ("moe_adapter_mm_dw", DW)):
        assert call(lib, fn, {**args, **small}, {}) == lib.MOE_ERR_WORKSPACE, fn


# ---------------------------------------------------------------- adapters
MM = dict(dtype=0, x=BUF, x_ld=128, a=BUF, a_l=16 * 128, a_r=128, b=BUF, b_l=128 * 16, b_n=16, offsets=BUF, order=BUF,
          scale=BUF, adapters=3, rows=10, N=128, K=128, rank=16, base=BUF + 4096, base_ld=128, out=BUF, out_ld=128, mid=BUF)
DW = dict(dtype=0, dy=BUF, dy_ld=128, x=BUF, x_ld=128, mid_x=BUF, mid_dy=BUF, offsets=BUF, order=BUF, scale=BUF,
          adapters=3, rows=10, N=128, K=128, rank=16, grad_dtype=2, accumulate=0, da=BUF, da_l=16 * 128, da_r=128,
          db=BUF, db_l=128 * 16, db_n=16)
SIZES = [dict(dtype=2), dict(dtype=-1), dict(adapters=0), dict(adapters=4097), dict(rows=-1), dict(rows=2 ** 31 - 1),
         dict(N=0), dict(K=0), dict(N=(1 << 21) + 1), dict(rank=0), dict(rank=257), dict(workspace=0),
         dict(workspace=BUF + 128), dict(offsets=0), dict(offsets=BUF + 2), dict(order=BUF + 2), dict(scale=BUF + 1)]


@pytest.mark.parametrize("bad", SIZES + [
    dict(x=0), dict(x=BUF + 1), dict(x_ld=127), dict(a=0), dict(a=BUF + 1), dict(a_l=-1), dict(a_r=127), dict(b=0),
    dict(b=BUF + 1), dict(b_l=-1), dict(b_n=15), dict(base=BUF + 1), dict(base_ld=127), dict(out=BUF + 1),
    dict(out_ld=127), dict(base=BUF, base_ld=136), dict(mid=BUF + 2), dict(out=0, mid=0)], ids=str)
@pytest.mark.parametrize("fn", ["moe_adapter_mm", "moe_adapter_mm_dx"])
def test_adapter_refusals(lib, fn, bad):
    assert call(lib, fn, {**MM, **workspace(lib)}, bad) == lib.MOE_ERR_INVALID


@pytest.mark.parametrize("fn", ["moe_adapter_mm", "moe_adapter_mm_dx"])
def test_adapter_mid_and_no_rows(lib, fn):
    assert call(lib, fn, {**MM, **workspace(lib)}, dict(mid=0, rows=(1 << 18) + 1)) == lib.MOE_ERR_WORKSPACE
    none = dict(rows=0, x=0, a=0, b=0, offsets=0, order=0, scale=0, base=0, out=0, mid=0)
    assert call(lib, fn, {**MM, **workspace(lib)}, none) == lib.MOE_OK


@pytest.mark.parametrize("bad", SIZES + [
    dict(dy=0), dict(dy=BUF + 1), dict(dy_ld=127), dict(x=0), dict(x=BUF + 1), dict(x_ld=127), dict(mid_x=0),
    dict(mid_x=BUF + 2), dict(mid_dy=0), dict(mid_dy=BUF + 2), dict(grad_dtype=1), dict(grad_dtype=3),
    dict(accumulate=2), dict(accumulate=1, grad_dtype=0), dict(da=BUF + 2), dict(da_r=127), dict(da_l=15 * 128 + 127),
    dict(db=BUF + 2), dict(db_n=15), dict(db_l=127 * 16 + 15)], ids=str)
def test_adapter_gradient_refusals(lib, bad):
    assert call(lib, "moe_adapter_mm_dw", {**DW, **workspace(lib)}, bad) == lib.MOE_ERR_INVALID


# ---------------------------------------------------------------- arguments in one array
def entries(lib):
    return (("moe_route", lib.route, ROUTE), ("moe_route_grad", lib.route_grad, ROUTE_GRAD),
            ("moe_expert_counts", lib.expert_counts, {**COUNTS, **workspace(lib)}),
            ("moe_balance_loss", lib.balance_loss, {**LOSS, **workspace(lib)}),
            ("moe_balance_loss_grad", lib.balance_loss_grad, {**LOSS_GRAD, **workspace(lib)}),
            ("moe_adapter_mm", lib.adapter_mm, {**MM, **workspace(lib)}),
            ("moe_adapter_mm_dx", lib.adapter_mm_dx, {**MM, **workspace(lib)}),
            ("moe_adapter_mm_dw", lib.adapter_mm_dw, {**DW, **workspace(lib)}))


def test_packed_arguments_arrive_in_their_places(lib):
    # Each argument made wrong on its own, so that nothing is launched: both ways give the entry's own answer.
    for fn, packed, args in entries(lib):
        for name in args:
            if name in ("scale", "stream", "order", "bias") and fn.startswith("moe_route"):
                continue
            bad = dict(args, **{name: -1 if name not in ("stream", "accumulate", "renormalize") else 2})
            if name == "stream":
                bad["rows" if "rows" in bad else "tokens"] = -1
            assert packed(*bad.values()) == call(lib, fn, bad, {}) in (lib.MOE_ERR_INVALID, lib.MOE_ERR_WORKSPACE), (fn, name)


def test_packed_calls_refuse(lib):
    import struct
    moe_call = lib.load().moe_call
    one = struct.pack("q", 0)
    for entry in (-1, 8, 1 << 20):
        assert moe_call(entry, one, 1) == lib.MOE_ERR_INVALID
    for entry, (fn, _, args) in enumerate(entries(lib)):
        n = len(args)
        values = struct.pack(f"{n + 1}q", *[0] * (n + 1))
        assert moe_call(entry, None, n) == lib.MOE_ERR_INVALID
        for count in (-1, 0, n - 1, n + 1):
            assert moe_call(entry, values, count) == lib.MOE_ERR_INVALID, (fn, count)


def test_no_fallback_on_the_cpu(lib):
    from weight_only_bit_moe_gb300 import adapters as A
    from weight_only_bit_moe_gb300 import routing as R
    x, a, b = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 3, 8, dtype=torch.bfloat16), torch.zeros(2, 5, 3, dtype=torch.bfloat16)
    off, ids, one = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.ones(())
    for f in (lambda: A.adapter_mm(x, a, b, off), lambda: A.adapter_mm_dx(x, a, b, off), lambda: A.adapter_linear(x, a, b, off),
              lambda: A.adapter_mm_dw(x, x, x.float(), x.float(), off), lambda: R.topk_route(x, 2), lambda: R.route(x, 2),
              lambda: R.topk_route_grad(ids.float(), x, ids), lambda: R.expert_counts(ids, 8),
              lambda: R.balance(x, ids[0]), lambda: R.balance_grad(one, x, ids[0])):
        with pytest.raises(ValueError, match="GPU"):
            f()


@pytest.mark.gpu
def test_python_refusals(lib):
    from gpu_util import need_gpu
    need_gpu()
    from weight_only_bit_moe_gb300 import adapters as A
    from weight_only_bit_moe_gb300 import routing as R
    bf, cu, i32 = torch.bfloat16, "cuda", torch.int32
    x, dy = torch.zeros(4, 8, dtype=bf, device=cu), torch.zeros(4, 5, dtype=bf, device=cu)
    a, b = torch.zeros(2, 3, 8, dtype=bf, device=cu), torch.zeros(2, 5, 3, dtype=bf, device=cu)
    off, order = torch.zeros(3, dtype=i32, device=cu), torch.arange(4, dtype=i32, device=cu)
    mid, scale = torch.zeros(4, 3, device=cu), torch.ones(2, device=cu)
    l, ids, one = torch.zeros(4, 6, device=cu), torch.zeros(4, 2, dtype=i32, device=cu), torch.ones((), device=cu)
    c = torch.zeros(6, dtype=i32, device=cu)
    bad = [
        lambda: A.adapter_mm(x.float(), a, b, off),
        lambda: A.adapter_mm(x.half(), a, b, off),
        lambda: A.adapter_mm(x[:, :7], a, b, off),
        lambda: A.adapter_mm(x.t().contiguous().t(), a, b, off),
        lambda: A.adapter_mm(x, a[0], b, off),
        lambda: A.adapter_mm(x, a, b[:1], off),
        lambda: A.adapter_mm(x, a, b[:, :, :2], off),
        lambda: A.adapter_mm(x, a.transpose(1, 2), b, off),
        lambda: A.adapter_mm(x, a, b, off[:2]),
        lambda: A.adapter_mm(x, a, b, off.long()),
        lambda: A.adapter_mm(x, a, b, off.cpu()),
        lambda: A.adapter_mm(x, a, b, off, order[:3]),
        lambda: A.adapter_mm(x, a, b, off, order.long()),
        lambda: A.adapter_mm(x, a, b, off, scale=scale.half()),
        lambda: A.adapter_mm(x, a, b, off, scale=scale[:1]),
        lambda: A.adapter_mm(x, a, b, off, base=x),
        lambda: A.adapter_mm(x, a, b, off, base=dy.float()),
        lambda: A.adapter_mm(x, a, b, off, out=dy[:3]),
        lambda: A.adapter_mm(x, a, b, off, out=dy.half()),
        lambda: A.adapter_mm(x, a, b, off, mid=mid[:, :2]),
        lambda: A.adapter_mm(x, a, b, off, mid=mid.half()),
        lambda: A.adapter_mm(x, torch.zeros(2, 257, 8, dtype=bf, device=cu), torch.zeros(2, 5, 257, dtype=bf, device=cu), off),
        lambda: A.adapter_mm_dx(x, a, b, off),
        lambda: A.adapter_mm_dw(dy, x[:3], mid, mid, off),
        lambda: A.adapter_mm_dw(dy, x, mid, None, off),
        lambda: A.adapter_mm_dw(None, None, None, None, off),
        lambda: A.adapter_mm_dw(dy, x, mid, mid[:, :2], off),
        lambda: A.adapter_mm_dw(dy, x, mid, mid, off, out_dtype=torch.float16),
        lambda: A.adapter_mm_dw(dy, x, mid, mid, off, accumulate=True),
        lambda: A.adapter_mm_dw(dy, x, mid, mid, off, out=(a, b), accumulate=True),
        lambda: A.adapter_mm_dw(dy, x, mid, mid, off, out=(b, a)),
        lambda: A.adapter_linear(x, a, b, off, scale=scale.clone().requires_grad_()),
        lambda: R.topk_route(l, 0),
        lambda: R.topk_route(l, 7),
        lambda: R.topk_route(torch.zeros(2, 64, device=cu), 33),
        lambda: R.topk_route(l.double(), 2),
        lambda: R.topk_route(l, 2, score="relu"),
        lambda: R.topk_route(l, 2, bias=c),
        lambda: R.topk_route(l, 2, bias=torch.zeros(5, device=cu)),
        lambda: R.topk_route(l.t(), 2),
        lambda: R.topk_route(l, 2, weights=mid),
        lambda: R.topk_route(l, 2, ids=ids.long()),
        lambda: R.topk_route(torch.zeros(2, 1025, device=cu), 2),
        lambda: R.topk_route_grad(mid, l, ids),
        lambda: R.topk_route_grad(mid[:, :2].half(), l, ids),
        lambda: R.topk_route_grad(mid[:, :2], l, ids.long()),
        lambda: R.topk_route_grad(mid[:, :2], l, ids, out=l.half()),
        lambda: R.expert_counts(ids.long(), 6),
        lambda: R.expert_counts(ids, 0),
        lambda: R.expert_counts(ids, 1025),
        lambda: R.expert_counts(ids, 6, off[:1]),
        lambda: R.expert_counts(ids, 6, off.long()),
        lambda: R.expert_counts(ids, 6, out=mid),
        lambda: R.balance(l, c.float()),
        lambda: R.balance(l, c[:5]),
        lambda: R.balance(l, c, off),
        lambda: R.balance_grad(one[None], l, c),
        lambda: R.balance_grad(one.double(), l, c),
        lambda: R.balance_grad(one, l, c, out=l[:3]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"refusal {i} was accepted")
