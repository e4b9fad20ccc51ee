"""Experts in three precisions, as one program uses them.

serve()  a layer whose routed experts are 4-bit (MoELayer) beside a shared expert in
         block-scaled FP8: quantise the tokens, gate and up projection, quantise
         silu(gate) * up, down projection.
experts_fp8()  routed experts in FP8: the tokens are gathered in expert order on their
         way through the quantisation, the products are grouped by expert.
tune()   routed experts in bf16 and their gradients: a few steps of gradient descent.

    python examples/mixed_precision_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from weight_only_bit_moe_gb300 import products as P  # noqa: E402
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


def relative(got, want):
    return float((got.float() - want).norm() / want.norm())


if __name__ == "__main__":
    _, mlp, want = serve()
    print(f"shared expert in FP8: relative error {relative(mlp, want):.4f}")
    out, want = experts_fp8()
    print(f"routed experts in FP8: relative error {relative(out, want):.4f}")
    print("tuning bf16 experts, loss by step: " + " ".join(f"{v:.4f}" for v in tune()))
    assert P.products_status() == 0
