"""Routing, counts and balance loss (include/moe_routing.h) against 64-bit references
on the GPU."""
import pytest
import torch

from gpu_util import need_gpu
from products_util import offsets_of
from tuning_util import (assert_bound, ref_balance, ref_route, ref_route_grad, rel_bound)

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


@pytest.fixture(scope="module")
def R():
    need_gpu()
    from weight_only_bit_moe_gb300 import routing
    return routing


@pytest.fixture(autouse=True)
def status():
    need_gpu()
    from weight_only_bit_moe_gb300 import products as P
    P.products_status()
    yield
    assert P.products_status() == 0


def make_logits(tokens, experts, dtype=torch.float32, seed=0, scale=1.5):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(tokens, experts, generator=g, device="cuda") * scale
            + torch.randn(experts, generator=g, device="cuda")).to(dtype)


def check_route(R, logits, top_k, score, bias, renormalize, scale):
    weights, ids = R.topk_route(logits, top_k, score, bias, renormalize, scale)
    want, want_ids = ref_route(logits, top_k, score, bias, renormalize, scale)
    assert torch.equal(ids, want_ids)
    assert_bound(weights, want, rel_bound(logits) * want.abs() + 2.0 ** -120, "weights")
    g = torch.Generator("cuda").manual_seed(3)
    dw = torch.randn(weights.shape, generator=g, device="cuda")
    check_grad(R, dw, logits, ids, score, renormalize, scale)
    return weights, ids


def check_grad(R, dw, logits, ids, score, renormalize, scale):
    got = R.topk_route_grad(dw, logits, ids, score, renormalize, scale)
    ref, mag = ref_route_grad(dw, logits, ids, score, renormalize, scale)
    assert_bound(got, ref, 4 * rel_bound(logits) * mag + 2.0 ** -120, "dlogits")


SIZES = [(1, 1, 1), (1, 2, 2), (5, 8, 2), (3, 7, 7), (17, 32, 4), (9, 33, 6), (130, 64, 8), (31, 100, 3), (77, 128, 8),
         (1000, 160, 6), (65, 256, 8), (12, 257, 32), (21, 384, 10), (40, 512, 8), (6, 513, 5), (33, 1024, 32),
         (4, 1021, 1)]


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(R, size, dtype):
    tokens, experts, top_k = size
    logits = make_logits(tokens, experts, dtype, seed=experts)
    bias = torch.randn(experts, device="cuda") * 0.1
    for score in ("softmax", "sigmoid"):
        check_route(R, logits, top_k, score, None, True, 1.0)
        check_route(R, logits, top_k, score, None, False, 2.5)
        check_route(R, logits, top_k, score, bias, True, 2.5)
        check_route(R, logits, top_k, score, bias, False, 1.0)


def test_many_tokens_with_a_bias(R):
    """Keys that 32 bits put in the wrong order or make equal, among some hundred thousand comparisons."""
    logits = make_logits(20000, 256, seed=1)
    bias = torch.randn(256, device="cuda") * 0.05
    for score in ("softmax", "sigmoid"):
        check_route(R, logits, 8, score, bias, True, 1.0)
    for top_k in (31, 32):  # as many as a warp has lanes: the next one decides too
        check_route(R, logits, top_k, "sigmoid", bias, True, 1.0)
    check_route(R, logits, 32, "softmax", None, False, 1.0)


def test_keys_next_to_each_other(R):
    """Pairs of experts whose score + bias differ by less than 32 bits resolve."""
    g = torch.Generator("cuda").manual_seed(2)
    l = torch.randn(500, 64, generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        p = torch.softmax(l.double(), 1) if score == "softmax" else torch.sigmoid(l.double())
        for t in range(0, 500, 50):
            bias = (0.5 - p[t]).float()  # every key of token t is 1/2 to within 2^-25
            check_route(R, l[t:t + 3].contiguous(), 8, score, bias, True, 1.0)


def test_equal_logits_go_by_number(R):
    logits = torch.tensor([[1.0, 2.0, 2.0, -0.0, 0.0, 2.0, 1.0, 0.0]], device="cuda")
    for dtype in DTYPES:
        for score in ("softmax", "sigmoid"):
            for bias in (None, torch.zeros(8, device="cuda")):
                _, ids = R.topk_route(logits.to(dtype), 8, score, bias)
                assert ids.tolist() == [[1, 2, 5, 0, 6, 3, 4, 7]]


@pytest.mark.parametrize("experts", [8, 40, 130, 1024])
def test_masked_experts(R, experts):
    top_k = 4
    logits = make_logits(40, experts)
    keep = torch.arange(experts, device="cuda")
    for t in range(40):  # token t keeps t % 7 experts
        mask = (keep * 5 + t) % experts >= t % 7
        logits[t, mask] = -INF
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.randn(experts, device="cuda") * 0.1):
            for renormalize in (True, False):
                weights, ids = check_route(R, logits, top_k, score, bias, renormalize, 1.5)
                for t in range(40):
                    n = min(top_k, int((logits[t] > -INF).sum()))
                    assert (ids[t] >= 0).sum() == n and (weights[t, n:] == 0).all()
    bias = torch.zeros(experts, device="cuda")
    bias[1:] = -INF
    w, ids = R.topk_route(make_logits(3, experts), 2, "sigmoid", bias)
    assert ids.tolist() == [[0, -1]] * 3 and w.tolist() == [[1.0, 0.0]] * 3


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(R, score):
    big = 3.0e38
    rows = [[big, -big, 0.0, 1.0], [-big, -big, -big, -big], [-200.0, -201.0, -300.0, -250.0], [200.0, 201.0, 199.0, 150.0],
            [88.0, 90.0, -88.0, -90.0], [-INF, -INF, 3.0, -INF], [-120.0, -120.0, -INF, -130.0]]
    logits = torch.tensor(rows, device="cuda")
    for renormalize in (True, False):
        for bias in (None, torch.tensor([0.0, 0.1, -0.1, 0.2], device="cuda")):
            w, ids = R.topk_route(logits, 3, score, bias, renormalize)
            want, want_ids = ref_route(logits, 3, score, bias, renormalize, 1.0)
            assert torch.equal(ids, want_ids)
            assert_bound(w, want, 2.0 ** -16 * want.abs() + 2.0 ** -126, "weights")
            d = R.topk_route_grad(torch.ones_like(w), logits, ids, score, renormalize)
            assert torch.isfinite(d).all()
    ids = R.topk_route(logits, 2, score)[1]
    check_balance(R, logits[2:], R.expert_counts(ids, 4), None, score)
    loss = R.balance(logits, R.expert_counts(ids, 4), None, score)
    assert torch.isfinite(loss) and torch.isfinite(R.balance_grad(torch.ones_like(loss), logits, R.expert_counts(ids, 4), None, score)).all()


@pytest.mark.parametrize("experts,top_k", [(16, 2), (40, 3), (40, 20), (300, 8), (1000, 32)])
def test_distances_past_the_largest_number(R, experts, top_k):
    """Experts so far below the largest that fp32 has no number for the distance still go by their own values."""
    g = torch.Generator("cuda").manual_seed(experts)
    far = -(1.0 + 2.3 * torch.rand(20, experts, generator=g, device="cuda")) * 1e38
    far[:, 7] = 3.3e38
    far[10:, 3] = 2e29
    for score in ("softmax", "sigmoid"):
        for logits, bias in ((far, None), (far, far[0] * 0.1), (far * 1e-38, far[0].contiguous()), (far, -far[1])):
            w, ids = R.topk_route(logits, top_k, score, bias)
            want, want_ids = ref_route(logits, top_k, score, bias, True, 1.0)
            assert torch.equal(ids, want_ids)
            assert_bound(w, want, 2.0 ** -16 * want.abs() + 2.0 ** -126, "weights")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinity_are_seen(R, score):
    logits = make_logits(6, 40)
    logits[1, 7], logits[3, 39], logits[4, 0] = float("nan"), INF, float("nan")
    logits[4, 1:] = -INF
    for bias in (None, torch.zeros(40, device="cuda")):
        w, ids = R.topk_route(logits, 4, score, bias)
        for t in range(6):
            if t in (1, 3, 4):
                assert torch.isnan(w[t]).all() and (ids[t] == -1).all()
            else:
                assert torch.isfinite(w[t]).all() and (ids[t] >= 0).all()
        d = R.topk_route_grad(torch.ones_like(w), logits, ids, score)
        assert (d[[1, 3, 4]] == 0).all()
    bias = torch.zeros(40, device="cuda")
    bias[2] = float("nan")
    w, ids = R.topk_route(logits, 4, score, bias)
    assert torch.isnan(w).all() and (ids == -1).all()


def test_gradient_for_other_ids(R):
    """Ids that the caller made: outside the experts, standing twice."""
    logits = make_logits(5, 24)
    ids = torch.tensor([[3, 3, 5], [-1, 2, 24], [-1, -7, 99], [0, 23, 0], [2 ** 31 - 1, 1, 1]], dtype=torch.int32, device="cuda")
    dw = torch.randn(5, 3, device="cuda")
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            check_grad(R, dw, logits, ids, score, renormalize, 1.7)
    bad = dw.clone()
    bad[1, 0] = float("nan")  # (of a slot without an expert)
    assert torch.isfinite(R.topk_route_grad(bad, logits, ids)).all()


@pytest.mark.parametrize("experts,pad", [(128, 4), (128, 3), (30, 2)])
def test_strides(R, experts, pad):
    big = torch.full((52, experts + pad), float("nan"), device="cuda")
    logits = make_logits(50, experts)
    view = big[1:51, :experts]
    view.copy_(logits)
    w, ids = R.topk_route(logits, 5)
    got = R.topk_route(view, 5)
    assert torch.equal(got[0], w) and torch.equal(got[1], ids)
    dw = torch.randn(50, 8, device="cuda")
    out = torch.full_like(big, 7.0)
    R.topk_route_grad(dw[:, :5], view, ids, out=out[1:51, :experts])
    assert torch.equal(out[1:51, :experts], R.topk_route_grad(dw[:, :5].contiguous(), logits, ids))
    assert (out[0] == 7).all() and (out[51] == 7).all() and (out[:, experts:] == 7).all()
    # balance
    counts = R.expert_counts(ids, experts)
    # (rows off the vectors' grid put other experts on a lane: sums in another order)
    check_balance(R, view, counts, None, "softmax")
    one = torch.ones((), device="cuda")
    out.fill_(7.0)
    R.balance_grad(one, view, counts, out=out[1:51, :experts])
    _, grad, mag = ref_balance(logits, counts[None], [0, 50], "softmax")
    rel = float(rel_bound(logits).max())
    assert_bound(out[1:51, :experts], grad, (4 * rel + (experts + 64) * 2.0 ** -23) * mag + 2.0 ** -120)
    assert (out[0] == 7).all() and (out[51] == 7).all() and (out[:, experts:] == 7).all()


def test_autograd_of_the_route(R):
    logits = make_logits(40, 48).requires_grad_()
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            w, ids = R.route(logits, 4, score, None, renormalize, 2.0)
            assert not ids.requires_grad
            g = torch.randn_like(w)
            got = torch.autograd.grad(w, logits, g)[0]
            assert torch.equal(got, R.topk_route_grad(g, logits.detach(), ids, score, renormalize, 2.0))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(R, score, renormalize):
    logits = make_logits(30, 16)
    w, ids = R.topk_route(logits, 4, score, None, renormalize)
    dw = torch.randn(w.shape, device="cuda")
    grad = R.topk_route_grad(dw, logits, ids, score, renormalize).double()
    d = torch.randn(logits.shape, device="cuda")
    h = 2.0 ** -7
    f = []
    for sign in (1, -1):  # the weights of the same experts, from the scores of moved logits
        p = logits + sign * h * d
        a, at = R.topk_route(p, 16, score, None, False)
        full = torch.zeros_like(p).scatter_(1, at.long(), a).double().gather(1, ids.long())
        f.append(full / full.sum(1, keepdim=True) if renormalize else full)
    left = (dw.double() * (f[0] - f[1])).sum(1) / (2 * h)
    right = (grad * d.double()).sum(1)
    # the third derivative of such weights is below 8 |d|^3; the values' own rounding is 2^-20 / h
    bound = dw.double().abs().sum(1) * (8 * (h * d.double().abs().sum(1)) ** 2 * d.double().abs().sum(1) / 6 + 2.0 ** -20 / h)
    assert ((left - right).abs() <= bound).all()


# ---------------------------------------------------------------- counts
@pytest.mark.parametrize("tokens,top_k,experts,lengths", [
    (1, 1, 1, None), (5, 2, 8, None), (123, 2, 8, None), (4096, 8, 128, None), (70000, 8, 256, None), (300, 3, 1024, None),
    (1000, 4, 64, [100, 0, 1, 399, 500]), (2000, 8, 128, [3] * 500), (50000, 6, 160, [20000, 0, 29000]), (64, 2, 16, [0])])
def test_counts(R, tokens, top_k, experts, lengths):
    g = torch.Generator("cuda").manual_seed(tokens)
    ids = torch.randint(-2, experts + 3, (tokens, top_k), generator=g, device="cuda", dtype=torch.int32)
    ids[::3] = 0 if experts > 0 else -1  # a popular one
    offsets = None if lengths is None else offsets_of(lengths)
    got = R.expert_counts(ids, experts, offsets)
    spans = [(0, tokens)] if lengths is None else list(zip(offsets.tolist()[:-1], offsets.tolist()[1:]))
    want = torch.stack([(ids[a:b].reshape(-1, 1) == torch.arange(experts, device="cuda")).sum(0) if b > a else
                        torch.zeros(experts, dtype=torch.int64, device="cuda") for a, b in spans]).to(torch.int32)
    assert torch.equal(got, want[0] if lengths is None else want)
    wide = torch.full((tokens, top_k + 3), 1, dtype=torch.int32, device="cuda")
    wide[:, :top_k] = ids
    assert torch.equal(R.expert_counts(wide[:, :top_k], experts, offsets), got)


def test_counts_of_no_tokens(R):
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert R.expert_counts(ids, 5).tolist() == [0] * 5
    assert R.expert_counts(ids, 3, offsets_of([0, 0])).tolist() == [[0] * 3] * 2


# ---------------------------------------------------------------- balance
def check_balance(R, logits, counts, offsets, score):
    loss = R.balance(logits, counts, offsets, score)
    S = 1 if offsets is None else len(offsets) - 1
    at = [0, logits.shape[0]] if offsets is None else offsets.tolist()
    ref, grad, mag = ref_balance(logits, counts.reshape(S, -1), at, score)
    rel = float(rel_bound(logits).max()) if logits.shape[0] else 0.0
    bound = (2 * rel + (logits.shape[1] + 64) * 2.0 ** -23) * ref.abs()
    assert_bound(loss.reshape(S), ref, bound, "loss")
    g = torch.Generator("cuda").manual_seed(8)
    dloss = torch.randn(S, generator=g, device="cuda")
    got = R.balance_grad(dloss.reshape(loss.shape), logits, counts, offsets, score)
    per = torch.zeros(logits.shape[0], dtype=torch.float64, device="cuda")
    for s in range(S):
        per[at[s]:at[s + 1]] = dloss[s].double()
    assert_bound(got, grad * per[:, None], (4 * rel + (logits.shape[1] + 64) * 2.0 ** -23) * mag * per.abs()[:, None] +
                 2.0 ** -120, "dlogits")
    return loss


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,lengths", [
    (1, 1, None), (1, 8, None), (123, 8, None), (50, 33, [10, 0, 1, 30]), (700, 128, None), (3000, 256, [1000, 7, 0, 1900]),
    (900, 160, [2] * 400), (40, 1024, [13, 20]), (20, 1000, None), (6, 40, [0, 0])])
def test_balance(R, tokens, experts, lengths, score, dtype):
    logits = make_logits(tokens, experts, dtype)
    ids = R.topk_route(logits, min(3, experts))[1]
    offsets = None if lengths is None else offsets_of(lengths)
    check_balance(R, logits, R.expert_counts(ids, experts, offsets), offsets, score)


def test_balance_of_many_tokens(R):
    logits = make_logits(40000, 128, torch.bfloat16)
    offsets = offsets_of([39000, 500])
    ids = R.topk_route(logits, 8)[1]
    a = check_balance(R, logits, R.expert_counts(ids, 128, offsets), offsets, "softmax")
    assert torch.equal(a, R.balance(logits, R.expert_counts(ids, 128, offsets), offsets))  # the same bits


def test_balance_of_even_counts_and_none(R):
    logits = make_logits(64, 16)
    assert abs(float(R.balance(logits, torch.full((16,), 5, dtype=torch.int32, device="cuda"))) - 1) < 1e-5
    none = torch.zeros(16, dtype=torch.int32, device="cuda")
    assert float(R.balance(logits, none)) == 0
    assert (R.balance_grad(torch.ones((), device="cuda"), logits, none) == 0).all()
    assert float(R.balance(logits[:0], none + 1)) == 0
    large = torch.full((16,), 2 ** 30, dtype=torch.int32, device="cuda")  # counts of many batches
    assert abs(float(R.balance(logits, large)) - 1) < 1e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_with_masked_experts(R, score):
    logits = make_logits(60, 40)
    logits[:, 5:9] = -INF
    logits[7] = -INF
    logits[9] = -150.0 - torch.arange(40, device="cuda")
    ids = R.topk_route(logits, 3)[1]
    check_balance(R, logits, R.expert_counts(ids, 40), None, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(R, score):
    logits = make_logits(50, 24)
    offsets = offsets_of([20, 25])
    counts = R.expert_counts(R.topk_route(logits, 3)[1], 24, offsets)
    leaf = logits.clone().requires_grad_()
    g = torch.tensor([0.7, -1.3], device="cuda")
    grad = torch.autograd.grad(R.balance_loss(leaf, counts, offsets, score), leaf, g)[0].double()
    assert torch.equal(grad, R.balance_grad(g, logits, counts, offsets, score).double())
    d = torch.randn(logits.shape, device="cuda")
    h = 2.0 ** -5
    f = [R.balance(logits + sign * h * d, counts, offsets, score).double() for sign in (1, -1)]
    left = float((g.double() * (f[0] - f[1])).sum()) / (2 * h)
    right = float((grad * d.double()).sum())
    # p's third derivative along d is below 26 max |d|^3 p-weighted; losses of a few, rounded to 2^-20
    bound = float((g.abs() * f[0].float().abs().clamp_min(1)).sum()) * (26 * h * h * float(d.abs().max()) ** 3 / 6 + 2.0 ** -20 / h)
    assert abs(left - right) <= bound


def test_broken_sequences_are_reported(R):
    from weight_only_bit_moe_gb300 import products as P
    logits = make_logits(50, 24)
    ids = R.topk_route(logits, 3)[1]
    counts = torch.ones(2, 24, dtype=torch.int32, device="cuda")
    for broken in ([-1, 20, 50], [0, 60, 50], [30, 20, 50], [0, 20, 51]):
        offsets = torch.tensor(broken, dtype=torch.int32, device="cuda")
        for call in (lambda: R.expert_counts(ids, 24, offsets), lambda: R.balance(logits, counts, offsets),
                     lambda: R.balance_grad(torch.ones(2, device="cuda"), logits, counts, offsets)):
            call()
            assert P.products_status() == P.B.MOE_ERR_INVALID


# ---------------------------------------------------------------- together, streams, graphs
def step(R, logits, top_k, offsets, dloss, dw):
    w, ids = R.topk_route(logits, top_k)
    counts = R.expert_counts(ids, logits.shape[1], offsets)
    loss = R.balance(logits, counts, offsets)
    return w, ids, counts, loss, R.balance_grad(dloss, logits, counts, offsets), R.topk_route_grad(dw, logits, ids)


def test_captured_and_on_another_stream(R):
    offsets = offsets_of([300, 100, 90])
    dloss, dw = torch.randn(3, device="cuda"), torch.randn(500, 4, device="cuda")
    logits, other = make_logits(500, 64), make_logits(500, 64, seed=4)
    want, want_other = step(R, logits, 4, offsets, dloss, dw), step(R, other, 4, offsets, dloss, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(R, logits, 4, offsets, dloss, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
    eager = step(R, other, 4, offsets, dloss, dw)  # at the same time
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(eager, want_other):
        assert torch.equal(a, b)
    logits.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want_other):
        assert torch.equal(a, b)
    for stream in (side, side.cuda_stream):
        w, ids = R.topk_route(other, 4, stream=stream)
        counts = R.expert_counts(ids, 64, offsets, stream=stream)
        loss = R.balance(other, counts, offsets, stream=stream)
        d = R.balance_grad(dloss, other, counts, offsets, stream=stream)
        side.synchronize()
        for a, b in zip((w, ids, counts, loss, d), want_other):
            assert torch.equal(a, b)


def test_captured_training_step(R):
    """Route, balance loss and adapters with their gradients in one graph, no eager graph of them left."""
    from weight_only_bit_moe_gb300 import adapters as A
    g = torch.Generator("cuda").manual_seed(5)

    def make(*shape):
        return (torch.randn(*shape, generator=g, device="cuda") * 0.2).to(torch.bfloat16)

    x, a, b = make(300, 64), make(2, 8, 64), make(2, 72, 8)
    logits, offsets = make_logits(300, 32), offsets_of([200, 90])

    def run():
        leaves = [t.detach().requires_grad_() for t in (x, a, b, logits)]
        y = A.adapter_linear(*leaves[:3], offsets)
        weights, ids = R.route(leaves[3], 4)
        loss = R.balance_loss(leaves[3], R.expert_counts(ids, 32, offsets), offsets)
        total = y.float().square().sum() + (weights * weights).sum() + loss.sum()
        return torch.autograd.grad(total, leaves)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in (x, a, b):
        t.copy_(make(*t.shape))
    logits.copy_(make_logits(300, 32, seed=9))
    graph.replay()
    torch.cuda.synchronize()
    for replayed, eager in zip(got, run()):
        assert torch.equal(replayed, eager)


def test_router_layer_adapters_together(R):
    """Router, 4-bit layer, an adapted FP8 projection and the balance loss in one step, with gradients."""
    from weight_only_bit_moe_gb300 import adapters as A
    from weight_only_bit_moe_gb300 import products as P
    from weight_only_bit_moe_gb300 import workloads as wk
    from weight_only_bit_moe_gb300.layer import MoELayer, batch_to_device
    wl = wk.WORKLOADS["tiny-int4"]
    layer = MoELayer.from_numpy(wk.make_weights(wl, 0))
    x, _, _, _ = batch_to_device(wk.make_batch(wl, 64, 1))
    g = torch.Generator("cuda").manual_seed(0)
    router = (torch.randn(wl.E, wl.K, generator=g, device="cuda") * wl.K ** -0.5).requires_grad_()
    logits = x.float() @ router.t()
    weights, ids = R.route(logits, 2)
    want, want_ids = ref_route(logits.detach(), 2, "softmax", None, True, 1.0)
    assert torch.equal(ids, want_ids)
    routed = layer(x, ids, weights.detach(), act=wl.act)
    assert torch.isfinite(routed).all()
    loss = R.balance_loss(logits, R.expert_counts(ids, wl.E)) + (weights * want.float()).sum()
    assert torch.isfinite(torch.autograd.grad(loss, router)[0]).all()
    # two tuned variants and plain requests on one FP8 projection
    codes = (torch.randn(96, wl.K, generator=g, device="cuda")).to(torch.float8_e4m3fn)
    scales = torch.full((1, -(-wl.K // 128)), 0.05, device="cuda")
    y = P.gemm_fp8_block(*P.quant_fp8_block(x), codes, scales)
    a = (torch.randn(2, 16, wl.K, generator=g, device="cuda") * wl.K ** -0.5).to(torch.bfloat16)
    b = torch.randn(2, 96, 16, generator=g, device="cuda").to(torch.bfloat16)
    who = torch.randint(-1, 2, (64, 1), generator=g, device="cuda")
    order, offsets = P.expert_order(who, 2)
    got = A.adapter_mm(x, a, b, offsets, order, base=y)
    for r in range(64):
        l = int(who[r])
        ref = y[r].double()
        if l >= 0:
            ref = ref + b[l].double() @ (a[l].double() @ x[r].double())
        assert torch.allclose(got[r].double(), ref, rtol=2.0 ** -7, atol=2.0 ** -6)
