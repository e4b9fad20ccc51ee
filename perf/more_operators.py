"""Routing, its balance loss and low-rank adapters as measured workloads.

* ``route``: the k best experts of each token's logits and their weights (softmax
  or sigmoid scores, with a selection bias, renormalised), alone or with the
  gradient by the logits;
* ``balance``: pairs per expert and sequence, the balance loss of each sequence
  and its gradient by the logits;
* ``adapter``: low-rank adapters of many requests added to a shared projection's
  output, alone or with the gradients by the rows and by both factors.

``run`` computes them in elementary torch operations, or with ``own`` set through
this package's entry points.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # a few decoding tokens: the call's latency
        dict(name="route-few", op="route", dtype="fp32", tokens=5, experts=32, top_k=4, score="softmax", bias=False,
             renormalize=True, scale=1.0, grad=False),
        # a prompt batch with sigmoid scores, a selection bias and a routed scale
        dict(name="route-prompt", op="route", dtype="fp32", tokens=8191, experts=256, top_k=8, score="sigmoid",
             bias=True, renormalize=True, scale=2.5, grad=False),
        # a tuning step: selection, weights and the gradient by the logits
        dict(name="route-step", op="route", dtype="bf16", tokens=32768, experts=128, top_k=8, score="softmax",
             bias=False, renormalize=False, scale=1.0, grad=True),
        # a small layer's batch as one sequence
        dict(name="balance-small", op="balance", dtype="fp32", tokens=123, experts=8, top_k=2, score="softmax",
             sequences=1),
        # a tuning step over ragged sequences with padding behind the last
        dict(name="balance-step", op="balance", dtype="bf16", tokens=65536, experts=128, top_k=8, score="softmax",
             sequences=17),
        # one token of a small projection: latency
        dict(name="adapter-one-token", op="adapter", kind="requests", dtype="bf16", tokens=1, adapters=8, requests=1,
             rank=16, n=1024, k=512, grad=False),
        # a decode batch, every request with an adapter of its own choice, some with none
        dict(name="adapter-decode", op="adapter", kind="requests", dtype="bf16", tokens=64, adapters=128, requests=64,
             rank=16, n=4096, k=4096, grad=False),
        # prompts of several requests beside decoding ones
        dict(name="adapter-prompt", op="adapter", kind="requests", dtype="bf16", tokens=8191, adapters=32, requests=23,
             rank=64, n=4096, k=4096, grad=False),
        # one adapter per expert of a small layer: forward and every gradient
        dict(name="adapter-step-small", op="adapter", kind="experts", dtype="bf16", tokens=246, adapters=8, requests=0,
             rank=8, n=1024, k=512, grad=True),
        # one adapter per expert in a tuning step, sizes off the powers of two
        dict(name="adapter-step-experts", op="adapter", kind="experts", dtype="fp16", tokens=8188, adapters=32,
             requests=0, rank=32, n=2880, k=2880, grad=True),
        # one adapter of a dense projection in a tuning step
        dict(name="adapter-step-dense", op="adapter", kind="experts", dtype="bf16", tokens=16384, adapters=1,
             requests=0, rank=16, n=4096, k=7168, grad=True),
    ]


def draw(rng):
    largest = [work(c) for c in listed()]
    top_bytes, top_flops = (max(w[key] for w in largest) for key in ("bytes", "flops"))

    def size(lo, hi, step):
        v = max(lo, round(lo * (hi / lo) ** rng.random() / step) * step)
        return v if v < 512 or v % 512 else v + step  # the listed cases have the round sizes

    while True:
        op = rng.choice(["route", "balance", "adapter", "adapter"])
        if op == "route":
            experts = size(8, 512, 1)
            score = rng.choice(["softmax", "sigmoid"])
            case = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=size(1, 32768, 1), experts=experts,
                        top_k=rng.randint(1, min(16, experts)), score=score, bias=rng.random() < 0.5,
                        renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), grad=rng.random() < 0.5)
        elif op == "balance":
            experts, tokens = size(8, 512, 1), size(64, 65536, 1)
            case = dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=tokens, experts=experts,
                        top_k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                        sequences=size(1, min(512, tokens // 8), 1))
        else:
            kind, tokens = rng.choice(["requests", "experts"]), size(1, 16384, 1)
            adapters = size(1, 128, 1)
            case = dict(op=op, kind=kind, dtype=rng.choice(["bf16", "fp16"]), tokens=tokens, adapters=adapters,
                        requests=rng.randint(1, min(tokens, 96)) if kind == "requests" else 0,
                        rank=size(8, 128, 8), n=size(256, 7168, 8), k=size(256, 7168, 8), grad=rng.random() < 0.5)
        w = work(case)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return case


def _cuts(rng, total, parts):
    """`total` cut into `parts` ragged lengths of at least one."""
    inner = np.sort(rng.choice(np.arange(1, total), parts - 1, replace=False)) if parts > 1 else np.zeros(0, np.int64)
    return np.diff(np.concatenate([[0], inner, [total]])).astype(np.int64)


def _adapter_rows(case, seed):
    """Adapter of each row, -1 for none."""
    rng = np.random.default_rng(seed)
    tokens, adapters = case["tokens"], case["adapters"]
    if case["kind"] == "experts":  # rows in expert order
        return np.sort(rng.integers(0, adapters, tokens))
    lengths = _cuts(rng, tokens, case["requests"])
    # adapters of unequal popularity; one request in eight runs without
    popular = rng.permutation(adapters)[(adapters * rng.random(len(lengths)) ** 2).astype(np.int64)]
    popular[rng.random(len(lengths)) < 0.125] = -1
    if (popular < 0).all():
        popular[0] = 0
    return np.repeat(popular, lengths)


def _sequence_lengths(case, seed):
    """Lengths of the sequences and the padding behind them."""
    rng = np.random.default_rng(seed)
    padding = case["tokens"] // 16 if case["sequences"] > 1 else 0
    return _cuts(rng, case["tokens"] - padding, case["sequences"]), padding


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)

    op, tokens, dtype = case["op"], case["tokens"], DTYPES[case["dtype"]]
    if op in ("route", "balance"):
        experts, top_k = case["experts"], case["top_k"]
        # experts of unequal popularity, as routers have them
        logits = (normal(tokens, experts, scale=1.5) + normal(experts, scale=0.7)).to(dtype)
        state = dict(op=op, logits=logits, score=case["score"], experts=experts, top_k=top_k)
        if op == "route":
            state.update(bias=normal(experts, scale=0.05) if case["bias"] else None, renormalize=case["renormalize"],
                         scale=case["scale"])
            state["dweights"] = normal(tokens, top_k, scale=0.02) if case["grad"] else None
            return state
        ids = torch.argsort(logits.float(), dim=1, descending=True)[:, :top_k].to(torch.int32).contiguous()
        lengths, padding = _sequence_lengths(case, seed)
        # gradients in fp16 come with a loss scale, or they would lie below its range
        loss_scale = 64.0 * tokens if dtype == torch.float16 else 1.0
        state.update(ids=ids, offsets=_offsets(lengths), lengths=lengths.tolist(), padding=padding,
                     dloss=normal(len(lengths), scale=0.01 * loss_scale))
        return state
    n, k, rank, adapters = case["n"], case["k"], case["rank"], case["adapters"]
    rows = _adapter_rows(case, seed)
    keys = np.where(rows < 0, adapters, rows)
    order = np.argsort(keys, kind="stable")
    counts = np.bincount(keys, minlength=adapters + 1)[:adapters]
    state = dict(op=op, counts=counts.tolist(), offsets=_offsets(counts),
                 order=None if case["kind"] == "experts" else torch.tensor(order, dtype=torch.int32, device="cuda"))
    state["x"] = (normal(tokens, k) * torch.exp(normal(k, scale=0.5))).to(dtype)
    state["a"] = normal(adapters, rank, k, dtype=dtype, scale=k ** -0.5)
    state["b"] = normal(adapters, n, rank, dtype=dtype, scale=0.25 * rank ** -0.5)
    state["scale"] = torch.full((adapters,), 2.0, device="cuda") * torch.exp(normal(adapters, scale=0.2))
    state["base"] = normal(tokens, n, dtype=dtype)
    state["dy"] = normal(tokens, n, dtype=dtype, scale=0.05) if case["grad"] else None
    return state


def _run_own(s):
    from weight_only_bit_moe_gb300 import adapters, routing

    if s["op"] == "route":
        how = dict(score=s["score"], renormalize=s["renormalize"], scale=s["scale"])
        weights, ids = routing.topk_route(s["logits"], s["top_k"], bias=s["bias"], **how)
        if s["dweights"] is None:
            return weights, ids
        return weights, ids, routing.topk_route_grad(s["dweights"], s["logits"], ids, **how)
    if s["op"] == "balance":
        counts = routing.expert_counts(s["ids"], s["experts"], offsets=s["offsets"])
        loss = routing.balance(s["logits"], counts, offsets=s["offsets"], score=s["score"])
        return counts, loss, routing.balance_grad(s["dloss"], s["logits"], counts, offsets=s["offsets"], score=s["score"])
    x, a, b, where = s["x"], s["a"], s["b"], dict(order=s["order"], scale=s["scale"])
    if s["dy"] is None:
        return adapters.adapter_mm(x, a, b, s["offsets"], base=s["base"], **where)
    t, dt = (torch.empty(x.shape[0], a.shape[1], device=x.device) for _ in range(2))
    y = adapters.adapter_mm(x, a, b, s["offsets"], base=s["base"], mid=t, **where)
    dx = adapters.adapter_mm_dx(s["dy"], a, b, s["offsets"], mid=dt, **where)
    return (y, dx, *adapters.adapter_mm_dw(s["dy"], x, t, dt, s["offsets"], **where))


def _log_sigmoid(v):
    return torch.clamp(v, max=0.0) - torch.log1p(torch.exp(-v.abs()))


def _softmax(v):
    e = torch.exp(v - v.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _run_route(s):
    logits, top_k, scale = s["logits"].float(), s["top_k"], s["scale"]
    softmax = s["score"] == "softmax"
    keys = logits
    if s["bias"] is not None:  # values next to each other decide: 64 bits
        wide = s["logits"].double()
        keys = (_softmax(wide) if softmax else torch.exp(_log_sigmoid(wide))) + s["bias"].double()
    ids = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :top_k]
    picked = logits.gather(1, ids)
    if s["renormalize"]:
        weights = scale * _softmax(picked if softmax else _log_sigmoid(picked))
    else:
        probs = _softmax(logits) if softmax else None
        weights = scale * (probs.gather(1, ids) if softmax else torch.exp(_log_sigmoid(picked)))
    if s["dweights"] is None:
        return weights, ids.to(torch.int32)
    g = s["dweights"]
    grad = torch.zeros_like(logits)
    if s["renormalize"]:
        d = weights * (g - (g * weights).sum(1, keepdim=True) / scale)
        if not softmax:
            d = d * torch.exp(_log_sigmoid(-picked))
        grad.scatter_(1, ids, d)
    elif softmax:
        grad.scatter_(1, ids, g)
        grad = scale * probs * (grad - (grad * probs).sum(1, keepdim=True))
    else:
        grad.scatter_(1, ids, g * weights * torch.exp(_log_sigmoid(-picked)))
    return weights, ids.to(torch.int32), grad.to(s["logits"].dtype)


def _run_balance(s):
    experts, lengths = s["experts"], s["lengths"]
    logits = s["logits"].float()
    counts, losses, grads = [], [], []
    for i, (l, ids) in enumerate(zip(logits.split(lengths + [s["padding"]]), s["ids"].split(lengths + [s["padding"]]))):
        if i == len(lengths):
            grads.append(torch.zeros_like(l))
            break
        c = torch.zeros(experts, dtype=torch.int64, device=l.device)
        c.index_add_(0, ids.reshape(-1).long(), torch.ones_like(ids, dtype=torch.int64).reshape(-1))
        factor = experts / (lengths[i] * ids.numel())
        if s["score"] == "softmax":
            p = slope = _softmax(l)
        else:
            v = torch.exp(_log_sigmoid(l))
            total = v.sum(1, keepdim=True)
            p, slope = v / total, v * torch.exp(_log_sigmoid(-l)) / total
        cf = c.float()
        inner = (p * cf).sum(1, keepdim=True)
        counts.append(c.to(torch.int32))
        losses.append((factor * inner.double().sum()).float())
        grads.append(s["dloss"][i] * factor * slope * (cf - inner))
    return torch.stack(counts), torch.stack(losses), torch.cat(grads).to(s["logits"].dtype)


def _run_adapter(s):
    x, a, b, base, dy = s["x"], s["a"], s["b"], s["base"], s["dy"]
    y = base.clone()
    if dy is not None:
        dx, da, db = torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
    start = 0
    for l, count in enumerate(s["counts"]):
        if count == 0:
            continue
        rows = slice(start, start + count) if s["order"] is None else s["order"][start:start + count].long()
        start += count
        a32, b32, scale = a[l].float(), b[l].float(), s["scale"][l]
        x32 = x[rows].float()
        t = x32 @ a32.t()
        y[rows] = (base[rows].float() + scale * (t @ b32.t())).to(base.dtype)
        if dy is not None:
            dy32 = dy[rows].float()
            dt = scale * (dy32 @ b32)
            dx[rows] = (dt @ a32).to(x.dtype)
            da[l] = (dt.t() @ x32).to(a.dtype)
            db[l] = (scale * (dy32.t() @ t)).to(b.dtype)
    return y if dy is None else (y, dx, da, db)


def run(state):
    if own:
        return _run_own(state)
    return {"route": _run_route, "balance": _run_balance, "adapter": _run_adapter}[state["op"]](state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapter":
        return _exact_adapter(s)
    l = s["logits"].double()
    sigmoid = 1.0 / (1.0 + torch.exp(-l))
    if case["op"] == "balance":
        counts, losses, grads = [], [], []
        p = torch.softmax(l, 1) if case["score"] == "softmax" else sigmoid / sigmoid.sum(1, keepdim=True)
        slope = p if case["score"] == "softmax" else p * (1.0 - sigmoid)
        at = 0
        for i, n in enumerate(s["lengths"]):
            c = (s["ids"][at:at + n].reshape(-1, 1) == torch.arange(case["experts"], device="cuda")).sum(0)
            inner = p[at:at + n] @ c.double()
            factor = case["experts"] / (n * float(c.sum()))
            counts.append(c.to(torch.int32))
            losses.append(inner.sum() * factor)
            grads.append(s["dloss"][i].double() * factor * slope[at:at + n] * (c.double()[None] - inner[:, None]))
            at += n
        grads.append(torch.zeros_like(l[at:]))
        return torch.stack(counts), torch.stack(losses), torch.cat(grads)
    scores = torch.softmax(l, 1) if case["score"] == "softmax" else sigmoid
    keys = l.clone() if s["bias"] is None else scores + s["bias"].double()
    ids = torch.empty(l.shape[0], case["top_k"], dtype=torch.int64, device="cuda")
    index = torch.arange(l.shape[1], device="cuda")
    for j in range(case["top_k"]):
        best = keys.amax(1, keepdim=True)
        ids[:, j] = torch.where(keys == best, index, l.shape[1]).amin(1)
        keys.scatter_(1, ids[:, j:j + 1], -float("inf"))
    chosen = scores.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(chosen[:, :1])
    weights = case["scale"] * chosen / total
    if s["dweights"] is None:
        return weights, ids.to(torch.int32)
    # by the scores first, then by the logits
    g = s["dweights"].double() * case["scale"]
    ds = g / total
    if case["renormalize"]:
        ds = ds - (g * chosen).sum(1, keepdim=True) / total ** 2
    dscores = torch.zeros_like(l).scatter_(1, ids, ds)
    if case["score"] == "softmax":
        grad = scores * dscores - scores * (scores * dscores).sum(1, keepdim=True)
    else:
        grad = dscores * sigmoid * (1.0 - sigmoid)
    return weights, ids.to(torch.int32), grad


def _exact_adapter(s):
    y = s["base"].double()
    grads = None
    if s["dy"] is not None:
        grads = [torch.zeros_like(s[name], dtype=torch.float64) for name in ("x", "a", "b")]
    ends = np.cumsum(s["counts"]).tolist()
    order = torch.arange(len(y), device="cuda") if s["order"] is None else s["order"].long()
    for l, (begin, end) in enumerate(zip([0] + ends[:-1], ends)):
        if begin == end:
            continue
        at = order[begin:end]
        xl, al = s["x"].index_select(0, at).double(), s["a"][l].double()
        bl = s["scale"][l].double() * s["b"][l].double()
        mid = torch.einsum("ik,rk->ir", xl, al)
        y.index_add_(0, at, torch.einsum("ir,nr->in", mid, bl))
        if grads is not None:
            dyl = s["dy"].index_select(0, at).double()
            dmid = torch.einsum("in,nr->ir", dyl, bl)
            grads[0].index_copy_(0, at, torch.einsum("ir,rk->ik", dmid, al))
            grads[1][l] = torch.einsum("ir,ik->rk", dmid, xl)
            grads[2][l] = torch.einsum("in,ir->nr", dyl, mid) * s["scale"][l].double()
    return y if grads is None else (y, *grads)


def work(case):
    """Inputs read once, outputs written once; factors of the adapters that got rows."""
    op, tokens = case["op"], case["tokens"]
    if op in ("route", "balance"):
        experts, top_k = case["experts"], case["top_k"]
        each = tokens * experts * SIZE[case["dtype"]]
        if op == "route":
            total = each + 8 * tokens * top_k + (4 * experts if case["bias"] else 0)
            if case["grad"]:
                total += 4 * tokens * top_k + each
            return dict(bytes=total, flops=(4 + 2 * top_k + (4 if case["grad"] else 0)) * tokens * experts)
        sequences = case["sequences"]
        return dict(bytes=2 * each + 4 * tokens * top_k + 4 * sequences * (experts + 2), flops=12 * tokens * experts)
    n, k, rank = case["n"], case["k"], case["rank"]
    rows = _adapter_rows(case, 0)
    own_rows, touched = int((rows >= 0).sum()), len(np.unique(rows[rows >= 0]))
    factors = touched * rank * (n + k) * 2
    total = 2 * (own_rows * k + 2 * tokens * n) + factors + 4 * tokens
    flops = 2 * own_rows * rank * (n + k)
    if case["grad"]:
        total += 2 * (tokens * n + tokens * k) + case["adapters"] * rank * (n + k) * 2
        flops *= 3
    return dict(bytes=total, flops=flops)
