"""Cases of the mixture block's operators: routing and its gradient, the products in 8-bit integers,
and the shared expert built of them.

`run` computes a case either in plain torch operations in 32 bits (own = False) or through this
package's kernels (own = True), on the same inputs."""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FLT_MAX = 3.4028234663852886e38


def listed():
    return [
        # routing: the router of the 384-expert block, one decoded token, fp32 logits
        dict(name="route one token", op="route", T=1, E=384, k=8, scoring="sigmoid", bias=True, groups=1,
             topk_group=1, renorm=True, scale=2.5, dtype="f32", masked=0),
        # a decode batch with the experts in groups, logits as a bf16 product leaves them
        dict(name="route grouped batch", op="route", T=200, E=256, k=8, scoring="sigmoid", bias=True, groups=8,
             topk_group=4, renorm=True, scale=2.5, dtype="bf16", masked=3),
        # a prompt of the same router
        dict(name="route prompt", op="route", T=8192, E=384, k=8, scoring="sigmoid", bias=True, groups=1,
             topk_group=1, renorm=True, scale=2.5, dtype="f32", masked=0),
        # training: gradient at the router's logits, sparse (only the chosen experts) ...
        dict(name="route gradient", op="route_backward", T=2048, E=384, k=8, scoring="sigmoid", renorm=True,
             scale=2.5, dtype="f32"),
        # ... and dense (softmax over all experts, not renormalised), an odd expert count, bf16
        dict(name="route gradient dense", op="route_backward", T=16384, E=257, k=6, scoring="softmax",
             renorm=False, scale=1.0, dtype="bf16"),
        # a projection at one decoded token: x is quantised per token, then multiplied
        dict(name="linear one token", op="linear", T=1, K=7168, N=4096, dtype="bf16", codes=False, residual=False),
        # a ragged product of ready codes (odd row counts, K off the tile, padded row strides)
        dict(name="product odd", op="linear", T=33, K=1003, N=1111, dtype="f16", codes=True, residual=False),
        # the shared expert's second product for a mid-sized batch, added to what is there, fp32
        dict(name="linear batch", op="linear", T=300, K=2048, N=7168, dtype="f32", codes=False, residual=True),
        # a prompt through a projection
        dict(name="linear prompt", op="linear", T=8192, K=7168, N=4096, dtype="bf16", codes=False, residual=False),
        # the shared expert beside the routed ones: a small decode batch, a large one, a prompt
        dict(name="mlp decode", op="mlp", T=16, H=7168, I=2048, dtype="bf16"),
        dict(name="mlp batch", op="mlp", T=512, H=7168, I=2048, dtype="bf16"),
        dict(name="mlp prompt", op="mlp", T=8192, H=7168, I=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "linear", "linear", "mlp"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "route":
        T, scoring = _log(rng, 1, 8192), rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([1, 1, 2, 4, 8])
        topk_group = rng.randint(1, groups)
        E = groups * _log(rng, 8, 512 // groups)
        k = rng.randint(1, min(16, topk_group * E // groups))
        return dict(op=op, T=T, E=E, k=k, scoring=scoring, bias=scoring == "sigmoid" and rng.random() < 0.7,
                    groups=groups, topk_group=topk_group, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype, masked=rng.choice([0, 0, 3]))
    if op == "route_backward":
        E = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 16, 16384), E=E, k=rng.randint(1, min(16, E)),
                    scoring=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype)
    if op == "linear":
        return dict(op=op, T=_log(rng, 1, 8192), K=_log(rng, 64, 7168), N=_log(rng, 64, 4096), dtype=dtype,
                    codes=rng.random() < 0.4, residual=rng.random() < 0.3)
    return dict(op=op, T=_log(rng, 1, 8192), H=8 * _log(rng, 32, 896), I=_log(rng, 128, 2048),
                dtype=rng.choice(["bf16", "f16"]))


# --------------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------------
def _weight(g, N, K):
    """Codes and channel scales of a [N, K] weight, laid out once: int8, rows on 16-byte boundaries."""
    q = torch.randint(-127, 128, (N, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda", generator=g)[:, :K]
    s = (0.5 + torch.rand(N, device="cuda", generator=g)) / (73.3 * math.sqrt(K))
    return q, s


def _activations(g, T, K, dtype):
    """Rows of different size with a few large channels, as activations have them."""
    x = torch.randn(T, K, device="cuda", generator=g) * torch.exp(torch.randn(T, 1, device="cuda", generator=g) * 0.5)
    x[:, torch.randint(0, K, (max(1, K // 512),), device="cuda", generator=g)] *= 4.0
    return x.to(dtype)


def _logits(c, g):
    x = torch.randn(c["T"], c["E"], device="cuda", generator=g) * 1.5
    if c.get("masked"):  # experts that are out of service
        x[:, torch.randperm(c["E"], device="cuda", generator=g)[:c["masked"]]] = -math.inf
    return x.to(DTYPES[c["dtype"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"c": c}
    if c["op"] == "route":
        s["logits"] = _logits(c, g)
        s["bias"] = 0.05 * torch.randn(c["E"], device="cuda", generator=g) if c["bias"] else None
    elif c["op"] == "route_backward":
        s["logits"] = _logits(c, g)
        r = dict(c, groups=1, topk_group=1)
        s["ids"], s["weights"] = _route(s["logits"], None, r)
        s["grad"] = torch.randn(c["T"], c["k"], device="cuda", generator=g)
    elif c["op"] == "linear":
        x = _activations(g, c["T"], c["K"], DTYPES[c["dtype"]])
        if c["codes"]:
            q, s["x_scale"] = _quantize(x.float())
            s["x"] = torch.zeros(c["T"], (c["K"] + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :c["K"]]
            s["x"].copy_(q)
        else:
            s["x"] = x
        s["w"], s["w_scale"] = _weight(g, c["N"], c["K"])
        s["residual"] = None
        if c["residual"]:
            s["residual"] = torch.randn(c["T"], c["N"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
    else:
        s["x"] = _activations(g, c["T"], c["H"], DTYPES[c["dtype"]])
        s["w13"], s["w13_scale"] = _weight(g, 2 * c["I"], c["H"])
        s["w2"], s["w2_scale"] = _weight(g, c["H"], c["I"])
        s["residual"] = torch.randn(c["T"], c["H"], device="cuda", generator=g).to(DTYPES[c["dtype"]])
    return s


# --------------------------------------------------------------------------------------------------
# plain forms, in 32 bits
# --------------------------------------------------------------------------------------------------
def _route(logits, bias, c):
    x = logits.float()
    out = torch.isnan(x) | (x == -math.inf)
    x = torch.where(out, -math.inf, x).clamp(max=FLT_MAX)
    if c["scoring"] == "sigmoid":
        value = score = torch.where(out, 0.0, 1.0 / (1.0 + torch.exp(-x)))
    else:
        top = x.amax(1, keepdim=True)
        value = torch.where(out, 0.0, torch.exp(x - torch.where(top == -math.inf, 0.0, top)))
        score = value / value.sum(1, keepdim=True).clamp(min=1e-38)
    if bias is not None:
        value = score + bias
    key = torch.where(out, -math.inf, x if bias is None else value)
    if c["groups"] > 1:
        T, E, G = x.shape[0], x.shape[1], c["groups"]
        best = torch.where(out, -math.inf, value).view(T, G, E // G).topk(min(2, E // G), dim=2).values
        first, rest = best[:, :, 0], best[:, :, 1:].sum(2)
        order = torch.where(rest == -math.inf, first, first + rest).sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order[:, :c["topk_group"]], True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, -math.inf)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    ids = ids[:, :c["k"]]
    w = torch.where(key[:, :c["k"]] == -math.inf, 0.0, score.gather(1, ids))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-38)
    return ids.int(), w * c["scale"]


def _route_backward(grad, logits, ids, weights, c):
    ids = ids.long()
    dot = (grad * weights).sum(1, keepdim=True)
    d = torch.zeros(logits.shape, device=logits.device)
    at = grad - dot / c["scale"] if c["renorm"] else grad
    if c["scoring"] == "sigmoid":
        at = at * (1.0 - 1.0 / (1.0 + torch.exp(-logits.gather(1, ids).float())))
    elif not c["renorm"]:
        e = torch.exp(logits.float() - logits.float().amax(1, keepdim=True))
        d = -(e / e.sum(1, keepdim=True)) * dot
    return d.scatter_add_(1, ids, weights * at).to(logits.dtype)


def _quantize(x):
    top = x.abs().amax(1, keepdim=True)
    return torch.round(x * (127.0 / top)), (top / 127.0).squeeze(1)


def _product(q, q_scale, w, w_scale):
    return q.float() @ w.float().t() * q_scale[:, None] * w_scale[None, :]


def _plain(s):
    c = s["c"]
    if c["op"] == "route":
        ids, w = _route(s["logits"], s["bias"], c)
        return {"ids": ids, "weights": w}
    if c["op"] == "route_backward":
        return _route_backward(s["grad"], s["logits"], s["ids"], s["weights"], c)
    if c["op"] == "linear":
        q, qs = (s["x"], s["x_scale"]) if c["codes"] else _quantize(s["x"].float())
        y = _product(q, qs, s["w"], s["w_scale"])
    else:
        gu = _product(*_quantize(s["x"].float()), s["w13"], s["w13_scale"])
        gate, up = gu[:, :c["I"]], gu[:, c["I"]:]
        y = _product(*_quantize(gate / (1.0 + torch.exp(-gate)) * up), s["w2"], s["w2_scale"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[c["dtype"]])


def run(state):
    if not own:
        return _plain(state)
    import w4a16_int4_mixture_gb300 as chord

    s, c = state, state["c"]
    if c["op"] == "route":
        ids, w = chord.moe_route(s["logits"], c["k"], bias=s["bias"], scoring=c["scoring"], n_group=c["groups"],
                                 topk_group=c["topk_group"], renormalize=c["renorm"], scale=c["scale"])
        return {"ids": ids, "weights": w}
    if c["op"] == "route_backward":
        return chord.moe_route_backward(s["grad"], s["logits"], s["ids"], s["weights"], scoring=c["scoring"],
                                        renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "linear":
        if c["codes"]:
            return chord.int8_matmul(s["x"], s["x_scale"], s["w"], s["w_scale"], residual=s["residual"],
                                     out_dtype=DTYPES[c["dtype"]])
        return chord.int8_linear(s["x"], s["w"], s["w_scale"], residual=s["residual"])
    return chord.int8_mlp(s["x"], s["w13"], s["w13_scale"], s["w2"], s["w2_scale"], residual=s["residual"])


# --------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# --------------------------------------------------------------------------------------------------
def work(case):
    c, z = case, SIZE[case["dtype"]]
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * z + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "route_backward":
        dense = c["scoring"] == "softmax" and not c["renorm"]
        read = c["E"] * z if dense else c["k"] * z if c["scoring"] == "sigmoid" else 0
        return {"bytes": c["T"] * (c["E"] * z + 12 * c["k"] + read),
                "flops": c["T"] * (4 * c["E"] if dense else 8 * c["k"])}
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        x = T * K + 4 * T if c["codes"] else T * K * z
        return {"bytes": x + N * K + 4 * N + T * N * z * (2 if c["residual"] else 1), "flops": 2 * T * K * N}
    T, H, I = c["T"], c["H"], c["I"]
    return {"bytes": 3 * T * H * z + 3 * H * I + 4 * (2 * I + H), "flops": 6 * T * H * I}


def _route64(logits, bias, c):
    """Ids and weights of every row, one group and one choice after another, in 64 bits."""
    x = logits.double()
    ok = ~(torch.isnan(x) | torch.isneginf(x))
    x = torch.minimum(x, torch.full_like(x, FLT_MAX))
    if c["scoring"] == "sigmoid":
        p = torch.sigmoid(x)
    else:
        p = torch.softmax(torch.where(ok, x, torch.full_like(x, -1e300)), 1)
    p = torch.where(ok, p, torch.zeros_like(p))
    rank = (p + bias.double()) if bias is not None else p
    low = torch.full_like(rank, -math.inf)
    rank = torch.where(ok, rank, low)
    T, E = x.shape
    G = c["groups"]
    size = E // G
    if G > 1:
        rows = rank.view(T, G, size)
        a = rows.max(2)
        b = rows.scatter(2, a.indices[:, :, None], -math.inf).max(2).values
        of_group = a.values + torch.where(torch.isneginf(b), torch.zeros_like(b), b)
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        for _ in range(c["topk_group"]):
            at = of_group.masked_fill(keep, -math.inf)
            left = torch.where(keep, 2, 1) * torch.arange(G, device=x.device) + torch.where(keep, G, 0)
            at = torch.where(at == at.max(1, keepdim=True).values, left, 3 * G).argmin(1)
            keep[torch.arange(T, device=x.device), at] = True
        rank = torch.where(keep[:, :, None].expand(T, G, size).reshape(T, E), rank, low)
    ids, vals = [], []
    free = torch.ones(T, E, dtype=torch.bool, device=x.device)
    number = torch.arange(E, device=x.device).expand(T, E)
    for _ in range(c["k"]):
        r = torch.where(free, rank, low)
        best = r.max(1, keepdim=True).values
        at = torch.where(free & (r == best), number, E).min(1).values
        ids.append(at)
        vals.append(torch.where(torch.isneginf(best[:, 0]), 0.0, p.gather(1, at[:, None])[:, 0]))
        free = free & (number != at[:, None])
    w = torch.stack(vals, 1)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, torch.ones_like(total)), torch.zeros_like(w))
    return w * c["scale"]


def _linear64(x, w, w_scale, codes_scale=None):
    if codes_scale is None:
        top = x.abs().max(1, keepdim=True).values
        q, qs = torch.round(127.0 * x / top), top / 127.0
    else:
        q, qs = x, codes_scale.double()[:, None]
    return torch.mm(q, w.double().t()) * (qs * w_scale.double()[None, :])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        # the ids rank scores of 32 bits, so near ties have no value in 64
        return {"ids": None, "weights": _route64(s["logits"], s["bias"], c)}
    if c["op"] == "route_backward":
        x = s["logits"].double().requires_grad_(True)
        p = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, 1)
        w = p.gather(1, s["ids"].long())
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (w * (c["scale"] * s["grad"].double())).sum().backward()
        return x.grad
    if c["op"] == "linear":
        y = _linear64(s["x"].double(), s["w"], s["w_scale"], s["x_scale"] if c["codes"] else None)
    else:
        gu = _linear64(s["x"].double(), s["w13"], s["w13_scale"])
        y = _linear64(torch.nn.functional.silu(gu[:, :c["I"]]) * gu[:, c["I"]:], s["w2"], s["w2_scale"])
    return y if s["residual"] is None else y + s["residual"].double()
