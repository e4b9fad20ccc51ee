"""The expert and block-scaled matrix products as measured workloads.

Five directions of three operators that run next to the 4-bit layer:

* products grouped by expert, rows of one expert contiguous and of any number
  (``fwd``: y = x W_e^T, ``dx``: dx = dy W_e, ``dw``: dW_e = dy_e^T x_e), for
  experts held in 16 bits and for tuning them;
* the product in FP8 (E4M3) with one scale per 1 x 128 of the activations and per
  128 x 128 of the weights (``fp8``), dense or grouped by expert;
* the quantisation that feeds it (``quant``): 1 x 128 blocks of rows, gathered by
  a row index or through the gated activation.

``run`` computes them in elementary fp32 torch operations, or with ``own`` set
through this package's entry points.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128
E4M3_MAX = 448.0


def listed():
    return [
        # one token of a small layer, two experts: the call's latency
        dict(name="fwd-one-token", op="fwd", dtype="bf16", experts=8, tokens=1, top_k=2, n=1024, k=512, zipf=False),
        # a decode batch over many experts: streams the touched experts' weights
        dict(name="fwd-decode", op="fwd", dtype="bf16", experts=128, tokens=16, top_k=8, n=4096, k=1536, zipf=True),
        # a prompt batch, skewed routing: large tiles with ragged ends
        dict(name="fwd-prompt", op="fwd", dtype="bf16", experts=128, tokens=4096, top_k=8, n=4096, k=1536, zipf=True),
        # gradient of the rows, small layer, few rows an expert
        dict(name="dx-small", op="dx", dtype="bf16", experts=8, tokens=123, top_k=2, n=1024, k=512, zipf=False),
        # gradient of the rows in a tuning step, sizes off the powers of two
        dict(name="dx-step", op="dx", dtype="fp16", experts=32, tokens=2047, top_k=4, n=2880, k=2880, zipf=False),
        # gradient of a small layer's weights, kept in their own type
        dict(name="dw-small", op="dw", dtype="bf16", experts=8, tokens=2304, top_k=2, n=1024, k=512, zipf=False, out="bf16"),
        # gradient of the weights in a tuning step, in fp32 for the optimizer
        dict(name="dw-step", op="dw", dtype="fp16", experts=32, tokens=2047, top_k=4, n=2880, k=2880, zipf=False, out="fp32"),
        # tokens gathered in expert order on their way into the FP8 product
        dict(name="quant-routed", op="quant", dtype="bf16", tokens=2048, top_k=8, k=4096, gated=False),
        # the gate and up halves of the first product on their way into the second
        dict(name="quant-gated", op="quant", dtype="fp16", tokens=4093, top_k=0, k=2880, gated=True),
        # a dense projection for a few decoding requests
        dict(name="fp8-decode", op="fp8", experts=0, tokens=5, top_k=1, n=4096, k=7168, zipf=False),
        # the same projection over a prompt
        dict(name="fp8-prompt", op="fp8", experts=0, tokens=8191, top_k=1, n=4096, k=7168, zipf=False),
        # experts in FP8, some hundred ragged rows each
        dict(name="fp8-experts", op="fp8", experts=32, tokens=1024, top_k=8, n=4096, k=4096, zipf=False),
    ]


def draw(rng):
    largest = [work(c) for c in listed()]
    top_bytes, top_flops = (max(w[key] for w in largest) for key in ("bytes", "flops"))

    def size(lo, hi, step):
        v = max(lo, round(lo * (hi / lo) ** rng.random() / step) * step)
        return v if v < 512 or v % 512 else v + step  # the listed cases have the round sizes

    while True:
        op = rng.choice(["fwd", "dx", "dw", "quant", "fp8"])
        case = dict(op=op, tokens=size(1, 8192, 1), top_k=rng.randint(1, 8))
        if op == "quant":
            gated = rng.random() < 0.5
            case.update(dtype=rng.choice(["bf16", "fp16"]), k=size(256, 7168, 8), gated=gated,
                        top_k=0 if gated else rng.randint(0, 8))
        elif op == "fp8":
            experts = rng.choice([0, size(4, 128, 1)])
            case.update(experts=experts, n=size(128, 7168, 8), k=size(256, 7168, 16), zipf=rng.random() < 0.5,
                        top_k=1 if experts == 0 else rng.randint(1, 4))
        else:
            case.update(dtype=rng.choice(["bf16", "fp16"]), experts=size(8, 128, 1), n=size(128, 4096, 8),
                        k=size(128, 4096, 8), zipf=rng.random() < 0.5)
            if op == "dw":
                case.update(out=rng.choice([case["dtype"], "fp32"]))
        w = work(case)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return case


def _rows_per_expert(case, seed):
    """Rows routed to each expert: every token picks top_k distinct experts."""
    experts, tokens, top_k = case["experts"], case["tokens"], case["top_k"]
    if experts == 0:
        return [tokens]
    rng = np.random.default_rng(seed)
    skew = -1.2 * np.log(1.0 + rng.permutation(experts)) if case["zipf"] else np.zeros(experts)
    keys = skew - np.log(-np.log(rng.random((tokens, experts))))
    picked = np.argpartition(-keys, top_k - 1, axis=1)[:, :top_k]
    return np.bincount(picked.reshape(-1), minlength=experts).tolist()


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _blocks(t, dim):
    """t with dimension `dim` padded by zeros to whole blocks and split into (blocks, BLOCK)."""
    length = t.shape[dim]
    pad = -length % BLOCK
    if pad:
        shape = list(t.shape)
        shape[dim] = pad
        t = torch.cat([t, t.new_zeros(shape)], dim)
    return t.unflatten(dim, (-1, BLOCK))


def _spread(scale, block_dims, shape):
    """One value per block, repeated over the block's elements."""
    for d in block_dims:
        scale = scale.repeat_interleave(BLOCK, d)
    return scale[tuple(slice(0, s) for s in shape)]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    op, k = case["op"], case["k"]
    if op == "quant":
        tokens, top_k = case["tokens"], case["top_k"]
        # channels of unequal size, as activations have them
        width = 2 * k if case["gated"] else k
        x = (normal(tokens, width) * torch.exp(normal(width, scale=0.7))).to(DTYPES[case["dtype"]])
        rows = None
        if top_k:
            rows = torch.randint(0, tokens, (tokens * top_k,), generator=gen, device="cuda", dtype=torch.int32)
        return dict(op=op, x=x, rows=rows, gated=case["gated"])
    n = case["n"]
    sizes = _rows_per_expert(case, seed)
    total = sum(sizes)
    if op == "fp8":
        experts = max(1, case["experts"])
        x = normal(total, k) * torch.exp(normal(k, scale=0.5))
        x_scale = _blocks(x, 1).abs().amax(2).clamp_min(1e-6) / E4M3_MAX
        xq = (x / _spread(x_scale, (1,), x.shape)).to(torch.float8_e4m3fn)
        del x
        wq = torch.empty(experts, n, k, dtype=torch.float8_e4m3fn, device="cuda")
        w_scale = torch.empty(experts, -(-n // BLOCK), -(-k // BLOCK), device="cuda")
        for e in range(experts):
            w = normal(n, k, scale=k ** -0.5)
            w_scale[e] = _blocks(_blocks(w, 1), 0).abs().amax((1, 3)).clamp_min(1e-8) / E4M3_MAX
            wq[e] = (w / _spread(w_scale[e], (0, 1), w.shape)).to(torch.float8_e4m3fn)
        if case["experts"] == 0:
            return dict(op=op, x=xq, x_scale=x_scale, w=wq[0], w_scale=w_scale[0], offsets=None, sizes=sizes)
        return dict(op=op, x=xq, x_scale=x_scale, w=wq, w_scale=w_scale, offsets=_offsets(sizes), sizes=sizes)
    dtype = DTYPES[case["dtype"]]
    state = dict(op=op, offsets=_offsets(sizes), sizes=sizes)
    if op in ("fwd", "dw"):
        state["x"] = normal(total, k, dtype=dtype)
    if op in ("dx", "dw"):
        state["dy"] = normal(total, n, dtype=dtype, scale=0.05)
    if op in ("fwd", "dx"):
        w = torch.empty(case["experts"], n, k, dtype=dtype, device="cuda")
        for e in range(case["experts"]):
            w[e] = normal(n, k, scale=k ** -0.5)
        state["w"] = w
    if op == "dw":
        state["out"] = DTYPES[case["out"]]
    return state


def _run_own(s):
    from weight_only_bit_moe_gb300 import products

    if s["op"] == "fwd":
        return products.grouped_mm(s["x"], s["w"], s["offsets"])
    if s["op"] == "dx":
        return products.grouped_mm_dx(s["dy"], s["w"], s["offsets"])
    if s["op"] == "dw":
        return products.grouped_mm_dw(s["dy"], s["x"], s["offsets"], out_dtype=s["out"])
    if s["op"] == "quant":
        return products.quant_fp8_block(s["x"], rows=s["rows"], gated=s["gated"])
    return products.gemm_fp8_block(s["x"], s["x_scale"], s["w"], s["w_scale"], offsets=s["offsets"])


def run(state):
    s = state
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quant":
        x = s["x"] if s["rows"] is None else s["x"][s["rows"]]
        v = x.float()
        if s["gated"]:
            gate, up = v.chunk(2, 1)
            v = gate / (1.0 + torch.exp(-gate)) * up
        scale = (_blocks(v, 1).abs().amax(2) / E4M3_MAX).clamp_min(2.0 ** -126)
        q = (v * _spread(1.0 / scale, (1,), v.shape)).to(torch.float8_e4m3fn)
        return q, scale
    sizes = s["sizes"]
    if op == "fp8":
        x = s["x"].float() * _spread(s["x_scale"], (1,), s["x"].shape)
        if s["offsets"] is None:
            w = s["w"].float() * _spread(s["w_scale"], (0, 1), s["w"].shape)
            return (x @ w.t()).to(torch.bfloat16)
        shape = s["w"].shape[1:]
        return torch.cat([xe @ (w.float() * _spread(ws, (0, 1), shape)).t()
                          for xe, w, ws in zip(x.split(sizes), s["w"], s["w_scale"])]).to(torch.bfloat16)
    if op == "fwd":
        return torch.cat([x.float() @ w.float().t() for x, w in zip(s["x"].split(sizes), s["w"])]).to(s["x"].dtype)
    if op == "dx":
        return torch.cat([dy.float() @ w.float() for dy, w in zip(s["dy"].split(sizes), s["w"])]).to(s["dy"].dtype)
    return torch.stack([(dy.float().t() @ x.float()).to(s["out"])
                        for dy, x in zip(s["dy"].split(sizes), s["x"].split(sizes))])


def _round_e4m3(v):
    """Nearest E4M3 value (ties to even mantissa) of doubles within +-448."""
    exponent = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(exponent - 3.0)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        v = s["x"].double()
        if s["rows"] is not None:
            v = v.index_select(0, s["rows"].long())
        if case["gated"]:
            k = case["k"]
            v = v[:, :k] * torch.sigmoid(v[:, :k]) * v[:, k:]
        scale = torch.stack([b.abs().amax(1) for b in v.split(BLOCK, 1)], 1) / E4M3_MAX
        q = torch.cat([_round_e4m3(b / scale[:, i:i + 1].clamp_min(2.0 ** -126))
                       for i, b in enumerate(v.split(BLOCK, 1))], 1)
        return q, scale
    ends = np.cumsum(s["sizes"]).tolist()
    spans = list(zip([0] + ends[:-1], ends))
    if op == "fp8":
        weights = s["w"] if case["experts"] else s["w"][None]
        scales = s["w_scale"] if case["experts"] else s["w_scale"][None]
        y = torch.zeros(ends[-1], case["n"], dtype=torch.float64, device="cuda")
        for (a, b), w, ws in zip(spans, weights, scales):
            if a == b:
                continue
            w64 = w.double()
            for i in range(ws.shape[0]):
                for j in range(ws.shape[1]):
                    w64[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= ws[i, j].double()
            x64 = torch.cat([block * s["x_scale"][a:b, j:j + 1].double()
                             for j, block in enumerate(s["x"][a:b].double().split(BLOCK, 1))], 1)
            y[a:b] = torch.einsum("mk,nk->mn", x64, w64)
        return y
    if op == "fwd":
        y = torch.zeros(ends[-1], case["n"], dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(spans):
            y[a:b] = torch.einsum("mk,nk->mn", s["x"][a:b].double(), s["w"][e].double())
        return y
    if op == "dx":
        y = torch.zeros(ends[-1], case["k"], dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(spans):
            y[a:b] = torch.einsum("mn,nk->mk", s["dy"][a:b].double(), s["w"][e].double())
        return y
    dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(spans):
        dw[e] = torch.einsum("mn,mk->nk", s["dy"][a:b].double(), s["x"][a:b].double())
    return dw


def work(case):
    """Inputs read once, outputs written once; weights of the experts that got rows."""
    op, k = case["op"], case["k"]
    if op == "quant":
        # every routed row is written; the tokens behind them are read once
        rows = case["tokens"] * max(1, case["top_k"])
        width = 2 * k if case["gated"] else k
        out = rows * (k + 4 * -(-k // BLOCK))
        return dict(bytes=case["tokens"] * width * 2 + out + 4 * case["tokens"] * case["top_k"], flops=4 * rows * k)
    n = case["n"]
    sizes = _rows_per_expert(case, 0)
    rows, touched = sum(sizes), sum(1 for m in sizes if m)
    flops = 2 * rows * n * k
    if op == "fp8":
        blocks = -(-k // BLOCK)
        return dict(bytes=rows * (k + 4 * blocks) + touched * (n * k + 4 * -(-n // BLOCK) * blocks) + 2 * rows * n,
                    flops=flops)
    if op == "dw":
        each = 4 if case["out"] == "fp32" else 2
        return dict(bytes=2 * rows * (n + k) + each * case["experts"] * n * k, flops=flops)
    return dict(bytes=2 * rows * (n + k) + 2 * touched * n * k, flops=flops)
