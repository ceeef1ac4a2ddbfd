"""Cases of the MoE layer's operators around the dispatch: the router and its
gradient, the experts' matrix products forwards and backwards, and the
gradient of the combine. Each can run in a plain form (elementary torch
operations in 32 bits, the router's choice in 64) or through the package.

A case is one call of one operator, ``case["op"]``:

    route        router logits -> topk_idx, topk_weights
    route_grad   d topk_weights -> d logits
    product      rows @ weight of their expert, with bias, activation, residual
    weight_grad  d weight (and d bias) of such a product
    combine_grad d y -> d expert rows, d topk_weights
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # one decoded token through the router of a 256-expert layer: latency only
        dict(name="route, one token", op="route", tokens=1, experts=256, topk=8, score="sigmoid",
             bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5,
             dtype="bf16", masked=0.0),
        # the largest batch of the benchmark, router logits in fp32, grouped choice with a
        # balancing bias, some tokens padding
        dict(name="route, 65536 tokens", op="route", tokens=65536, experts=256, topk=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5, dtype="f32", masked=0.05),
        # training step of a small layer
        dict(name="route_grad, small", op="route_grad", tokens=64, experts=16, topk=2,
             score="sigmoid", renorm=True, scale=1.0, dtype="f32"),
        # training step, weights of a softmax over all experts: the gradient is dense
        dict(name="route_grad, 16384 tokens", op="route_grad", tokens=16384, experts=256, topk=8,
             score="softmax", renorm=False, scale=1.0, dtype="bf16"),
        # decode: 64 routed rows over the 8 experts of a rank; the weights' bytes are the cost
        dict(name="product, decode", op="product", experts=8, rows=64, k=7168, n=4096,
             act="swiglu", bias=False, residual=False, pre=False, transposed=False, out="bf16",
             spread="uniform", spare=0),
        # 2048 tokens, top-6 of 64 experts: bytes and operations in balance, whole epilogue
        dict(name="product, 64 experts", op="product", experts=64, rows=12288, k=4096, n=2048,
             act="gelu", bias=True, residual=True, pre=False, transposed=False, out="bf16",
             spread="uniform", spare=0),
        # receive side: 32768 rows over a rank's 8 experts, gated, training (z is kept)
        dict(name="product, 32768 rows", op="product", experts=8, rows=32768, k=7168, n=4096,
             act="swiglu", bias=False, residual=False, pre=True, transposed=False, out="bf16",
             spread="uniform", spare=0),
        # data gradient through the second product into the gated activation, uneven experts
        dict(name="product, data gradient", op="product", experts=8, rows=12289, k=7168, n=2048,
             act="swiglu_grad", bias=False, residual=False, pre=True, transposed=True,
             out="bf16", spread="skew", spare=511),
        # weight gradients of 64 experts with about 192 rows each, kept in fp32, with the bias'
        dict(name="weight_grad, 64 experts", op="weight_grad", experts=64, rows=12288, k=4096,
             n=2048, bias=True, out="f32", spread="uniform"),
        # the receive side's weight gradients: one large product over the rows of each expert
        dict(name="weight_grad, 29765 rows", op="weight_grad", experts=8, rows=29765, k=7168,
             n=4096, bias=False, out="bf16", spread="skew"),
        # the smallest batch of the benchmark
        dict(name="combine_grad, small", op="combine_grad", tokens=64, hidden=128, topk=2,
             dropped=0.1, dtype="f32"),
        # the benchmark's own batch
        dict(name="combine_grad, 4096 tokens", op="combine_grad", tokens=4096, hidden=7168,
             topk=8, dropped=0.0, dtype="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "product", "product", "weight_grad", "combine_grad"])
    if op in ("route", "route_grad"):
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        case = dict(op=op, tokens=_spread(rng, 1, 32768), experts=experts,
                    topk=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["f32", "bf16"]))
        case["renorm"] &= case["topk"] > 1       # a lone weight is always one
        if op == "route":
            groups = rng.choice([1, 1, 4, 8]) if experts >= 16 and experts % 8 == 0 else 1
            case.update(bias=rng.random() < 0.6, groups=groups,
                        topk_groups=groups if groups == 1 else rng.randint(groups // 2, groups),
                        group_top=rng.choice([1, 2]), masked=rng.choice([0.0, 0.1]))
        return case
    if op == "combine_grad":
        return dict(op=op, tokens=_spread(rng, 1, 4096), hidden=8 * _spread(rng, 16, 896),
                    topk=rng.randint(1, 8), dropped=rng.choice([0.0, 0.1, 0.8]),
                    dtype=rng.choice(["f32", "bf16"]))
    while True:
        experts = rng.choice([1, 2, 8, 16, 64])
        rows = _spread(rng, 1, 16384)
        k = 8 * _spread(rng, 8, 896)
        n = 16 * _spread(rng, 4, 256)
        if experts * k * n <= 64 * 4096 * 2048 and rows * k * n <= 16384 * 7168 * 2048:
            break
    spread = rng.choice(["uniform", "skew"])
    if op == "weight_grad":
        return dict(op=op, experts=experts, rows=rows, k=k, n=n, bias=rng.random() < 0.5,
                    out=rng.choice(["f32", "bf16"]), spread=spread)
    act = rng.choice(["none", "silu", "gelu", "swiglu", "silu_grad", "gelu_grad", "swiglu_grad"])
    grad = act.endswith("_grad")
    return dict(op=op, experts=experts, rows=rows, k=k, n=n, act=act,
                bias=not grad and rng.random() < 0.5, residual=not grad and rng.random() < 0.4,
                pre=grad or (act != "none" and rng.random() < 0.4),
                transposed=rng.random() < (0.7 if grad else 0.2),
                out=rng.choice(["bf16", "bf16", "f32"]), spread=spread,
                spare=rng.choice([0, 0, 37]))


_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _share(case, gen, dev):
    """How many rows each expert has, and where its block starts (int32)."""
    e = case["experts"]
    odds = torch.ones(e, device=dev)
    if case["spread"] == "skew":
        # a few experts get most rows
        odds = 1.0 / torch.arange(1, e + 1, device=dev, dtype=torch.float32).sqrt()
        odds = odds[torch.randperm(e, generator=gen, device=dev)]
    edges = torch.cumsum(odds / odds.sum(), 0)[:-1].contiguous()
    ids = torch.bucketize(torch.rand(case["rows"], generator=gen, device=dev), edges)
    counts = torch.bincount(ids, minlength=e)
    starts = torch.cumsum(counts, 0) - counts
    return counts.int(), starts.int()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype).mul_(std)

    s = {"case": dict(case)}
    op = case["op"]
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = normal(t, e, dtype=torch.float32, std=1.5).to(_DTYPE[case["dtype"]])
        if op == "route":
            s["bias"] = normal(e, std=0.05) if case["bias"] else None
            s["mask"] = (torch.rand(t, generator=gen, device=dev) >= case["masked"]).to(
                torch.uint8) if case["masked"] else None
        else:
            # the choice that the forward pass made, some slots empty
            order = torch.rand(t, e, generator=gen, device=dev).argsort(dim=1)[:, :k]
            empty = torch.rand(t, k, generator=gen, device=dev) < (0.02 if t > 64 else 0.0)
            s["idx"] = order.masked_fill(empty, -1).contiguous()
            s["grad"] = normal(t, k)
        return s
    if op == "combine_grad":
        t, h, k = case["tokens"], case["hidden"], case["topk"]
        empty = torch.rand(t * k, generator=gen, device=dev) < case["dropped"]
        place = torch.randperm(t * k, generator=gen, device=dev).int()
        s["index"] = place.masked_fill(empty, -1).view(t, k)
        s["weights"] = torch.rand(t, k, generator=gen, device=dev)
        s["rows"] = normal(t * k, h, dtype=torch.bfloat16)
        s["dy"] = normal(t, h).to(_DTYPE[case["dtype"]])
        s["out"] = torch.zeros(t * k, h, dtype=torch.bfloat16, device=dev)
        return s
    e, rows, k, n = case["experts"], case["rows"], case["k"], case["n"]
    s["counts"], s["starts"] = _share(case, gen, dev)
    s["longest"] = int(s["counts"].max())     # a program that pads knows how far
    total = rows + case.get("spare", 0)       # a buffer's capacity
    s["x"] = normal(total, k, dtype=torch.bfloat16)
    if op == "weight_grad":
        s["d"] = normal(total, n, dtype=torch.bfloat16)
        s["dw"] = torch.zeros(e, n, k, dtype=_DTYPE[case["out"]], device=dev)
        s["db"] = torch.zeros(e, n, device=dev) if case["bias"] else None
        return s
    act = case["act"]
    std = 1.0 / math.sqrt(k)
    s["w"] = normal(*((e, k, n) if case["transposed"] else (e, n, k)), dtype=torch.bfloat16,
                    std=std)
    s["b"] = normal(e, n, std=0.5) if case["bias"] else None
    cols = n // 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    s["res"] = normal(total, cols, dtype=torch.bfloat16) if case["residual"] else None
    s["y"] = torch.zeros(total, cols, dtype=_DTYPE[case["out"]], device=dev)
    s["pre"] = None
    if act.endswith("_grad"):
        s["pre"] = normal(total, cols, dtype=torch.bfloat16)
    elif case["pre"]:
        s["pre"] = torch.zeros(total, n, dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------ plain forms --

def _plain_route(c, s):
    x = s["logits"].double()       # the choice in 64 bits: neighbours may be close
    t, e = x.shape
    if c["score"] == "softmax":
        p = torch.exp(x - x.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        by_group = choice.view(t, c["groups"], -1)
        best = by_group.sort(dim=2, descending=True, stable=True).values[:, :, :c["group_top"]]
        order = best.sum(2).sort(dim=1, descending=True, stable=True).indices
        keep = torch.zeros(t, c["groups"], dtype=torch.bool, device=x.device)
        keep.scatter_(1, order[:, :c["topk_groups"]], True)
        choice = torch.where(keep[:, :, None], by_group, -math.inf).view(t, e)
    idx = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    if s["mask"] is not None:
        live = s["mask"][:, None] != 0
        idx = torch.where(live, idx, -1)
        w = torch.where(live, w, 0.0)
    return idx, w.float()


def _plain_route_grad(c, s):
    x, idx = s["logits"].float(), s["idx"]
    live = idx >= 0
    at = idx.clamp(min=0)
    if c["score"] == "softmax":
        p = torch.exp(x - x.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    chosen = torch.where(live, p.gather(1, at), 0.0)
    g = torch.where(live, s["grad"], 0.0) * c["scale"]
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        share = chosen / total
        g = (g - (share * g).sum(1, keepdim=True)) / total
        g = torch.where(live, g, 0.0)
    dp = torch.zeros_like(p).scatter_add_(1, at, g)
    if c["score"] == "softmax":
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        dx = dp * p * (1.0 - p)
    return dx.to(s["logits"].dtype)


def _blocks(s, total):
    """Places of each expert's rows in a rectangle [experts, longest], and back."""
    n = s["longest"]
    at = torch.arange(max(n, 1), device=s["counts"].device)
    live = at < s["counts"][:, None]
    place = (s["starts"][:, None] + at).clamp(max=total - 1).long()
    row = torch.arange(total, device=at.device)
    ends = (s["starts"] + s["counts"]).long()
    expert = torch.searchsorted(ends, row, right=True)
    used = expert < len(ends)
    expert = expert.clamp(max=len(ends) - 1)
    return live, place, used, expert, (row - s["starts"].long()[expert]).clamp(min=0, max=max(n, 1) - 1)


def _silu_gelu(act, z):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _slope(act, z):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
        z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)


def _plain_product(c, s):
    act = c["act"]
    total = s["x"].shape[0]
    live, place, used, expert, slot = _blocks(s, total)
    x = torch.where(live[:, :, None], s["x"][place].float(), 0.0)
    w = s["w"].float()
    z = torch.bmm(x, w if c["transposed"] else w.transpose(1, 2))
    z = z[expert, slot]
    if s["b"] is not None:
        z = z + s["b"][expert]
    if act == "none":
        y = z
    elif act == "swiglu":
        half = z.shape[1] // 2
        y = _silu_gelu("silu", z[:, :half]) * z[:, half:]
    elif act == "swiglu_grad":
        half = z.shape[1]
        gate, up = s["pre"][:, :half].float(), s["pre"][:, half:].float()
        y = torch.cat([z * up * _slope("silu", gate), z * _silu_gelu("silu", gate)], 1)
    elif act.endswith("_grad"):
        y = z * _slope(act[:4], s["pre"].float())
    else:
        y = _silu_gelu(act, z)
    if s["res"] is not None:
        y = y + s["res"].float()
    y = torch.where(used[:, None], y.to(s["y"].dtype), s["y"])
    if s["pre"] is None or act.endswith("_grad"):
        return y
    return y, torch.where(used[:, None], z.to(torch.bfloat16), s["pre"])


def _plain_weight_grad(c, s):
    live, place, *_ = _blocks(s, s["x"].shape[0])
    x = torch.where(live[:, :, None], s["x"][place].float(), 0.0)
    d = torch.where(live[:, :, None], s["d"][place].float(), 0.0)
    dw = torch.bmm(d.transpose(1, 2).contiguous(), x).to(s["dw"].dtype)
    return dw if s["db"] is None else (dw, d.sum(1))


def _plain_combine_grad(c, s):
    index, k = s["index"].long(), c["topk"]
    live = index >= 0
    dy = s["dy"].float()
    rows = s["rows"][index.clamp(min=0)].float()
    dw = torch.where(live, (rows * dy[:, None, :]).sum(2), 0.0)
    n = s["rows"].shape[0]
    slot = torch.full((n + 1,), -1, dtype=torch.long, device=dy.device)
    slot[torch.where(live, index, n).view(-1)] = torch.arange(index.numel(), device=dy.device)
    slot = slot[:n]
    at = slot.clamp(min=0)
    d = s["weights"].view(-1)[at][:, None] * dy[at // k]
    return torch.where(slot[:, None] >= 0, d.to(torch.bfloat16), s["out"]), dw


_PLAIN = {"route": _plain_route, "route_grad": _plain_route_grad, "product": _plain_product,
          "weight_grad": _plain_weight_grad, "combine_grad": _plain_combine_grad}


# -------------------------------------------------- the package's operators --

def _own_route(epl, c, s):
    return epl.route(s["logits"], c["topk"], score=c["score"], bias=s["bias"],
                     num_groups=c["groups"], topk_groups=c["topk_groups"],
                     group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"],
                     token_mask=s["mask"])


def _own_route_grad(epl, c, s):
    return epl.route_backward(s["logits"], s["idx"], s["grad"], score=c["score"],
                              renormalize=c["renorm"], scale=c["scale"])


def _own_product(epl, c, s):
    y = epl.expert_product(s["x"], s["w"], s["starts"], s["counts"], bias=s["b"],
                           activation=c["act"], residual=s["res"], pre=s["pre"], out=s["y"],
                           transposed=c["transposed"], expected_rows=c["rows"])
    return y if s["pre"] is None or c["act"].endswith("_grad") else (y, s["pre"])


def _own_weight_grad(epl, c, s):
    epl.expert_weight_grad(s["d"], s["x"], s["starts"], s["counts"], out=s["dw"],
                           bias_grad=s["db"])
    return s["dw"] if s["db"] is None else (s["dw"], s["db"])


def _own_combine_grad(epl, c, s):
    return epl.combine_backward(s["dy"], s["rows"], s["index"], s["weights"], grad_rows=s["out"])


_OWN = {"route": _own_route, "route_grad": _own_route_grad, "product": _own_product,
        "weight_grad": _own_weight_grad, "combine_grad": _own_combine_grad}


def run(state):
    c = state["case"]
    if own:
        import permute_ep_layout_amd as epl
        return _OWN[c["op"]](epl, c, state)
    return _PLAIN[c["op"]](c, state)


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["topk"]
        size = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": t * (e * size + k * 12 + (1 if case["masked"] else 0)) +
                    (4 * e if case["bias"] else 0), "flops": 10 * t * e}
        # only a softmax over all experts needs more than the chosen logits
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": t * (e * size + k * 12 + (e if dense else k) * size),
                "flops": 6 * t * e}
    if op == "combine_grad":
        t, h, k = case["tokens"], case["hidden"], case["topk"]
        slots = t * k * (1.0 - case["dropped"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": t * h * size + slots * h * 4 + t * k * 12, "flops": 3 * slots * h}
    e, rows, k, n = case["experts"], case["rows"], case["k"], case["n"]
    flops = 2.0 * rows * k * n
    size = 2 if case["out"] == "bf16" else 4
    if op == "weight_grad":
        out = e * n * (k * size + (4 if case["bias"] else 0))
        return {"bytes": rows * (k + n) * 2 + out,
                "flops": flops + (rows * n if case["bias"] else 0)}
    used = e * (1.0 - (1.0 - 1.0 / e) ** rows)        # experts with at least one row
    act = case["act"]
    cols = n / 2 if act == "swiglu" else 2 * n if act == "swiglu_grad" else n
    return {"bytes": 2 * (rows * k + used * n * k) + rows * cols * size +
            (4 * used * n if case["bias"] else 0) + (2 * rows * cols if case["residual"] else 0) +
            (2 * rows * (cols if act.endswith("_grad") else n) if case["pre"] else 0),
            "flops": flops + 10 * rows * n}


# ------------------------------------------- definitions, in 64 bits --

def _exact_route(c, s):
    x = s["logits"].cpu().double().numpy()
    t, e = x.shape
    if c["score"] == "softmax":
        p = np.exp(x - x.max(axis=1)[:, None])
        p /= p.sum(axis=1)[:, None]
    else:
        p = np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))),
                     np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))
    key = p.copy()
    if s["bias"] is not None:
        key += s["bias"].cpu().double().numpy()
    g, size = c["groups"], e // c["groups"]
    if g > 1:
        rank = np.stack([np.sort(key[:, i * size:(i + 1) * size], axis=1)[:, -c["group_top"]:].sum(
            axis=1) for i in range(g)], axis=1)
        gone = np.argsort(-rank, axis=1, kind="stable")[:, c["topk_groups"]:]
        for j in range(gone.shape[1]):
            for i in range(size):
                key[np.arange(t), gone[:, j] * size + i] = -np.inf
    idx = np.argsort(-key, axis=1, kind="stable")[:, :c["topk"]]
    w = np.take_along_axis(p, idx, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1)[:, None]
    w = w * c["scale"]
    if s["mask"] is not None:
        off = s["mask"].cpu().numpy() == 0
        idx[off], w[off] = -1, 0.0
    return idx, w


def _exact_route_grad(c, s):
    x = s["logits"].double()
    idx = s["idx"]
    one = torch.nn.functional.one_hot(idx.clamp(min=0), x.shape[1]).double()
    one = one * (idx >= 0)[:, :, None]                        # [tokens, topk, experts]
    if c["score"] == "softmax":
        p = torch.softmax(x, 1)
        slope = None
    else:
        p = torch.sigmoid(x)
        slope = torch.sigmoid(x) * torch.sigmoid(-x)
    grad = s["grad"].double() * c["scale"]
    s_k = (one * p[:, None, :]).sum(2)
    if c["renorm"]:
        d = s_k.sum(1, keepdim=True)
        d = torch.where(d > 0, d, torch.ones_like(d))
        grad = grad / d - (grad * s_k).sum(1, keepdim=True) / d ** 2
    dp = (one * grad[:, :, None]).sum(1)
    if slope is None:
        return p * dp - p * (p * dp).sum(1, keepdim=True)
    return dp * slope


def _each(s):
    """(expert, first row, last row + 1) of the experts that have rows."""
    for e, (n, at) in enumerate(zip(s["counts"].tolist(), s["starts"].tolist())):
        if n:
            yield e, at, at + n


def _exact_product(c, s):
    act = c["act"]
    y = s["y"].double()
    keeps = s["pre"] is not None and not act.endswith("_grad")
    pre = s["pre"].double() if keeps else None
    for e, a, b in _each(s):
        w = s["w"][e].double()
        z = s["x"][a:b].double() @ (w if c["transposed"] else w.t())
        if s["b"] is not None:
            z += s["b"][e].double()
        if keeps:
            pre[a:b] = z
        kept = s["pre"][a:b].double() if act.endswith("_grad") else None
        if act == "none":
            v = z
        elif act == "silu":
            v = z * torch.sigmoid(z)
        elif act == "gelu":
            v = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
        elif act == "swiglu":
            gate, up = z.chunk(2, 1)
            v = gate * torch.sigmoid(gate) * up
        elif act == "silu_grad":
            p = torch.sigmoid(kept)
            v = z * (p + kept * p * torch.sigmoid(-kept))
        elif act == "gelu_grad":
            v = z * (0.5 * torch.erfc(-kept / math.sqrt(2.0)) +
                     kept * torch.exp(-kept.square() / 2) * 0.3989422804014327)
        else:
            gate, up = kept.chunk(2, 1)
            p = torch.sigmoid(gate)
            v = torch.cat([z * up * (p + gate * p * torch.sigmoid(-gate)), z * gate * p], 1)
        if s["res"] is not None:
            v = v + s["res"][a:b].double()
        y[a:b] = v
    return (y, pre) if keeps else y


def _exact_weight_grad(c, s):
    dw = s["dw"].double()
    db = None if s["db"] is None else s["db"].double()
    for e, a, b in _each(s):
        d = s["d"][a:b].double()
        dw[e] = d.t() @ s["x"][a:b].double()
        if db is not None:
            db[e] = d.sum(0)
    return dw if db is None else (dw, db)


def _exact_combine_grad(c, s):
    out = s["out"].double()
    dw = torch.zeros(s["index"].shape, dtype=torch.float64, device=out.device)
    dy = s["dy"].double()
    for k in range(c["topk"]):
        at = s["index"][:, k].long()
        t = torch.nonzero(at >= 0)[:, 0]
        out[at[t]] = s["weights"][t, k].double()[:, None] * dy[t]
        dw[t, k] = (s["rows"][at[t]].double() * dy[t]).sum(1)
    return out, dw


_EXACT = {"route": _exact_route, "route_grad": _exact_route_grad, "product": _exact_product,
          "weight_grad": _exact_weight_grad, "combine_grad": _exact_combine_grad}


def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))
