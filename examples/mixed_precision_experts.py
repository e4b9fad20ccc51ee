"""Experts in three precisions, as one program uses them.

serve()  a layer whose routed experts are 4-bit (MoELayer) beside a shared expert in
         block-scaled FP8: quantise the tokens, gate and up projection, quantise
         silu(gate) * up, down projection.
experts_fp8()  routed experts in FP8: the tokens are gathered in expert order on their
         way through the quantisation, the products are grouped by expert.
tune()   routed experts in bf16 and their gradients: a few steps of gradient descent.
tune_adapters()  frozen experts with a low-rank adapter each, behind a router that is trained
         with them: the outputs, the balance loss and every gradient.
serve_adapters()  one FP8 projection for requests that each bring an adapter, or none.

    python examples/mixed_precision_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_bit_moe_gb300 import adapters as A  # noqa: E402
from weight_only_bit_moe_gb300 import products as P  # noqa: E402
from weight_only_bit_moe_gb300 import routing as R  # noqa: E402
from weight_only_bit_moe_gb300 import workloads as wk  # noqa: E402
from weight_only_bit_moe_gb300.layer import MoELayer, batch_to_device  # noqa: E402


def fp8_weights(w: torch.Tensor):
    """(E4M3 codes, fp32 scales) of a matrix or bank [..., N, K], one scale per 128 x 128."""
    n, k = w.shape[-2:]
    pad = torch.nn.functional.pad(w.float(), (0, -k % P.BLOCK, 0, -n % P.BLOCK))
    blocks = pad.unflatten(-1, (-1, P.BLOCK)).unflatten(-3, (-1, P.BLOCK))  # [..., N/128, 128, K/128, 128]
    scale = blocks.abs().amax((-3, -1)).clamp_min(2.0 ** -126) / 448.0
    codes = (blocks / scale[..., :, None, :, None]).flatten(-4, -3).flatten(-2, -1)
    return codes[..., :n, :k].to(torch.float8_e4m3fn).contiguous(), scale


def fp8_mlp(q, s, w13, w2, offsets=None):
    """Down(silu(gate) * up) of quantised rows; w13, w2: (codes, scales)."""
    h = P.gemm_fp8_block(q, s, *w13, offsets)
    q, s = P.quant_fp8_block(h, gated=True)
    return P.gemm_fp8_block(q, s, *w2, offsets)


def combine(y, order, topk_weights):
    """Rows in expert order -> tokens, weighted by their routing."""
    tokens, top_k = topk_weights.shape
    pairs = torch.zeros(tokens * top_k, y.shape[1], dtype=torch.float32, device=y.device)
    pairs[order.long()] = y.float()
    return (pairs.view(tokens, top_k, -1) * topk_weights[:, :, None]).sum(1)


def serve(tokens=64, shared=256, seed=0):
    """Layer output of 4-bit routed experts plus an FP8 shared expert, and the shared expert's part."""
    wl = wk.WORKLOADS["tiny-int4"]
    layer = MoELayer.from_numpy(wk.make_weights(wl, seed))
    x, ids, w, _ = batch_to_device(wk.make_batch(wl, tokens, seed + 1))
    g = torch.Generator("cuda").manual_seed(seed)
    w13 = torch.randn(2 * shared, wl.K, generator=g, device="cuda") * wl.K ** -0.5
    w2 = torch.randn(wl.K, shared, generator=g, device="cuda") * shared ** -0.5
    routed = layer(x, ids, w, act=wl.act)
    mlp = fp8_mlp(*P.quant_fp8_block(x), fp8_weights(w13), fp8_weights(w2))
    h = x.float() @ w13.t()
    want = (torch.nn.functional.silu(h[:, :shared]) * h[:, shared:]) @ w2.t()
    return routed + mlp, mlp, want


def experts_fp8(tokens=96, experts=8, top_k=2, hidden=512, inter=256, seed=0):
    """Output of routed FP8 experts and the same in fp32."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    w13 = torch.randn(experts, 2 * inter, hidden, generator=g, device="cuda") * hidden ** -0.5
    w2 = torch.randn(experts, hidden, inter, generator=g, device="cuda") * inter ** -0.5
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    weights, ids = torch.topk(torch.softmax(logits, 1), top_k)
    order, offsets = P.expert_order(ids, experts)
    q, s = P.quant_fp8_block(x, rows=order // top_k)
    out = combine(fp8_mlp(q, s, fp8_weights(w13), fp8_weights(w2), offsets), order, weights)
    h = torch.einsum("tk,enk->ten", x.float(), w13)
    a = torch.nn.functional.silu(h[..., :inter]) * h[..., inter:]
    y = torch.einsum("ten,ekn->tek", a, w2)
    want = (y.gather(1, ids[:, :, None].expand(-1, -1, hidden)) * weights[:, :, None]).sum(1)
    return out, want


def tune(steps=8, tokens=192, experts=4, top_k=2, hidden=256, inter=128, rate=0.2, seed=0):
    """Losses of gradient descent on bf16 experts that learn another set's outputs."""
    g = torch.Generator("cuda").manual_seed(seed)

    def bank(n, k):
        return (torch.randn(experts, n, k, generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16)

    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.topk(torch.rand(tokens, experts, generator=g, device="cuda"), top_k).indices
    order, offsets = P.expert_order(ids, experts)
    rows = x[(order // top_k).long()]

    def experts_out(w13, w2):
        gate, up = P.grouped_linear(rows, w13, offsets).chunk(2, 1)
        return P.grouped_linear(torch.nn.functional.silu(gate) * up, w2, offsets)

    with torch.no_grad():
        target = experts_out(bank(2 * inter, hidden), bank(hidden, inter)).float()
    masters = [bank(2 * inter, hidden).float(), bank(hidden, inter).float()]
    losses = []
    for _ in range(steps):
        params = [m.to(torch.bfloat16).requires_grad_() for m in masters]
        loss = (experts_out(*params).float() - target).square().mean()
        loss.backward()
        losses.append(float(loss.detach()))
        for m, p in zip(masters, params):
            m -= rate * tokens * p.grad.float()
    return losses


def tune_adapters(tokens=160, experts=4, top_k=2, hidden=256, inter=128, rank=8, seed=0):
    """One step's leaves (router, a, b), the objective's gradients by them and, from fp32, the same."""
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    x = normal(tokens, hidden).to(torch.bfloat16)
    w = normal(experts, inter, hidden, scale=hidden ** -0.5).to(torch.bfloat16)  # frozen
    leaves = [normal(experts, hidden, scale=hidden ** -0.5), normal(experts, rank, hidden, scale=hidden ** -0.5).to(torch.bfloat16),
              normal(experts, inter, rank, scale=rank ** -0.5).to(torch.bfloat16)]
    scale = torch.full((experts,), 2.0, device="cuda")
    router, a, b = (t.requires_grad_() for t in leaves)

    logits = x.float() @ router.t()
    weights, ids = R.route(logits, top_k)
    balance = R.balance_loss(logits, R.expert_counts(ids, experts))
    order, offsets = P.expert_order(ids, experts)
    rows = x[(order // top_k).long()]
    h = A.adapter_linear(rows, a, b, offsets, scale=scale, base=P.grouped_mm(rows, w, offsets))
    objective = combine(h, order, weights).square().mean() + 0.01 * balance
    grads = torch.autograd.grad(objective, (router, a, b))

    router, a, b = (t.detach().float().requires_grad_() for t in leaves)
    logits = x.float() @ router.t()
    p = torch.softmax(logits, 1)
    picked = torch.softmax(logits.gather(1, ids.long()), 1)
    counts = torch.bincount(ids.flatten().long(), minlength=experts).float()
    balance = experts * (counts / counts.sum() * p.mean(0)).sum()
    full = torch.einsum("tk,enk->ten", x.float(), w.float())
    full = full + 2.0 * torch.einsum("tk,erk,enr->ten", x.float(), a, b)
    out = (full.gather(1, ids.long()[:, :, None].expand(-1, -1, inter)) * picked[:, :, None]).sum(1)
    want = torch.autograd.grad(out.square().mean() + 0.01 * balance, (router, a, b))
    return leaves, grads, want


def serve_adapters(requests=24, adapters=6, hidden=512, out=384, rank=16, seed=0):
    """Outputs of one FP8 projection with each request's adapter, and the same in fp32."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(requests, hidden, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(out, hidden, generator=g, device="cuda") * hidden ** -0.5
    a = (torch.randn(adapters, rank, hidden, generator=g, device="cuda") * hidden ** -0.5).to(torch.bfloat16)
    b = (torch.randn(adapters, out, rank, generator=g, device="cuda") * rank ** -0.5).to(torch.bfloat16)
    who = torch.randint(-1, adapters, (requests, 1), generator=g, device="cuda")
    order, offsets = P.expert_order(who, adapters)  # once for all projections of a step
    y = P.gemm_fp8_block(*P.quant_fp8_block(x), *fp8_weights(w))
    A.adapter_mm(x, a, b, offsets, order, base=y, out=y)
    delta = torch.einsum("tk,lrk,lnr->tln", x.float(), a.float(), b.float())
    delta = torch.cat([torch.zeros_like(delta[:, :1]), delta], 1)  # number -1: none
    want = x.float() @ w.t() + delta[torch.arange(requests, device="cuda"), who[:, 0] + 1]
    return y, want


def relative(got, want):
    return float((got.float() - want).norm() / want.norm())


if __name__ == "__main__":
    _, mlp, want = serve()
    print(f"shared expert in FP8: relative error {relative(mlp, want):.4f}")
    out, want = experts_fp8()
    print(f"routed experts in FP8: relative error {relative(out, want):.4f}")
    print("tuning bf16 experts, loss by step: " + " ".join(f"{v:.4f}" for v in tune()))
    _, grads, want = tune_adapters()
    print("adapters and router, relative errors of the gradients: " + " ".join(f"{relative(g, w):.4f}" for g, w in zip(grads, want)))
    print(f"adapters of many requests on an FP8 projection: relative error {relative(*serve_adapters()):.4f}")
    assert P.products_status() == 0
