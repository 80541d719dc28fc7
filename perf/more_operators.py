"""Cases of a feed-forward layer's operators around the products, dense and routed.

A case's ``op`` names the operator, its ``grad`` the direction:

* ``fused``    c = act(A B^T + bias) + residual; gradient: dz = dy act'(z), dbias = column sums of dz
* ``route``    logits -> ids of the experts of each token and their gates; gradient: dlogits from dgates
* ``combine``  y[t] = residual[t] + sum_f gates[t, f] rows[inverse[t, f]]; gradient: drows and dgates

With ``own`` false the operators are computed in elementary torch operations in
32 bits, rounded once at the end; with it true by the library.
"""
import math

import torch

own = False


# ---- the cases --------------------------------------------------------------

def _fused(name, rows, n, k, act, bias, residual, pre=False, f32=False):
    return {"name": name, "op": "fused", "grad": False, "rows": rows, "n": n, "k": k, "act": act, "bias": bias,
            "residual": residual, "pre": pre, "f32": f32}


def _route(name, grad, tokens, experts, fan, score, bias, groups, top_groups, group_top, renormalize, scale, f32):
    return {"name": name, "op": "route", "grad": grad, "tokens": tokens, "experts": experts, "fan": fan, "score": score,
            "bias": bias, "groups": groups, "top_groups": top_groups, "group_top": group_top, "renormalize": renormalize,
            "scale": scale, "f32": f32}


def _combine(name, grad, tokens, fan, n, experts, dropped, residual, f32, out_f32):
    return {"name": name, "op": "combine", "grad": grad, "tokens": tokens, "fan": fan, "n": n, "experts": experts,
            "dropped": dropped, "residual": residual, "f32": f32, "out_f32": out_f32}


def listed():
    return [
        # one request decodes: the latency of a projection with its activation
        _fused("projection, one token", 1, 4096, 4096, "silu", "f16", False),
        # 48 requests decode together: the second projection of a block, onto the residual stream
        _fused("projection, decode", 48, 4096, 4096, "none", "f16", True),
        # 16384 tokens of a training step or a long prompt through the first projection; z is kept for the backward pass
        _fused("first projection, training", 16384, 4096, 2048, "gelu_tanh", "f32", False, pre=True),
        # the second projection of a block, onto the residual stream
        _fused("second projection, residual", 4096, 4096, 4096, "none", "f16", True),
        # a router's logits: few columns, in fp32, every token read once
        _fused("router's logits", 16384, 64, 4096, "none", "", False, f32=True),
        # no size a multiple of a tile, everything in the epilogue
        _fused("projection, ragged", 5000, 3000, 1000, "gelu", "f32", True),
        # the training step's gradient through the activation, with the bias's
        {"name": "activation gradient", "op": "fused", "grad": True, "rows": 16384, "n": 4096, "act": "gelu_tanh", "bias_grad": True},
        # a decoding step of 64 sequences, two of eight experts each
        _route("routing, decode", False, 64, 8, 2, "softmax", False, 1, 1, 1, True, 1.0, True),
        # a training batch: eight of 256 experts, at most four of eight groups, a bias that balances the load
        _route("routing, training", False, 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, True),
        # its backward pass, for softmax scores
        _route("routing gradient", True, 16384, 256, 8, "softmax", False, 1, 1, 1, True, 1.0, True),
        # 8192 tokens, two experts each: the experts' rows back onto the residual stream
        _combine("combination", False, 8192, 2, 4096, 8, 0.02, True, False, False),
        # its backward pass
        _combine("combination gradient", True, 8192, 2, 4096, 8, 0.02, False, False, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A matrix width: mostly whole 16-byte chunks, one in five any size."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.2 else max(8, v // 8 * 8)


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def draw(rng):
    op = rng.choice(["fused", "fused", "fused", "fused_grad", "route", "route", "route_grad", "combine", "combine_grad"])
    if op == "fused":
        n, k = _width(rng, 16, 4096), _width(rng, 64, 4096)
        rows = min(_log(rng, 1, 16384), 16384 * 4096 * 2048 // (n * k))
        case = _fused("", rows, n, k, rng.choice(ACTS), rng.choice(["", "f16", "f32"]), rng.random() < 0.5,
                      rng.random() < 0.3, rng.random() < 0.25)
    elif op == "fused_grad":
        case = {"op": "fused", "grad": True, "rows": _log(rng, 1, 16384), "n": _width(rng, 16, 4096), "act": rng.choice(ACTS),
                "bias_grad": rng.random() < 0.7}
        if case["act"] == "none":
            case["bias_grad"] = True
    elif op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 4, 256 // groups)
        top_groups = rng.randint(1, groups)
        fan = min(rng.choice([1, 2, 2, 4, 6, 8]), experts // groups * top_groups)
        case = _route("", op == "route_grad", _log(rng, 1, 16384), experts, fan, rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, top_groups, rng.choice([1, 2]), rng.random() < 0.7,
                      rng.choice([1.0, 1.0, 2.5]), rng.random() < 0.7)
        if case["grad"] and fan == 1:  # a single renormalised gate is constant: nothing to learn from
            case["renormalize"] = False
    else:
        fan, n = rng.choice([1, 2, 2, 4, 6, 8]), _width(rng, 64, 4096)
        tokens = min(_log(rng, 1, 16384), 8192 * 2 * 4096 // (2 * fan * n))
        f32 = rng.random() < 0.3
        case = _combine("", op == "combine_grad", tokens, fan, n, rng.choice([8, 16, 64]), rng.choice([0.0, 0.02, 0.2]),
                        rng.random() < 0.5, f32, rng.random() < 0.3)
    case.pop("name", None)
    return case


# ---- inputs -----------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, f32=False):
        t = torch.randn(*shape, generator=gen, device=dev) * std
        return t if f32 else t.to(torch.float16)

    s = dict(case)
    if case["op"] == "fused":
        rows, n = case["rows"], case["n"]
        if case["grad"]:
            s["dy"] = normal(rows, n, std=0.125)
            s["z"] = normal(rows, n, std=1.5) if case["act"] != "none" else None
            return s
        k = case["k"]
        s["a"] = normal(rows, k)
        s["b"] = normal(n, k, std=k ** -0.5)
        s["bias_t"] = normal(n, std=0.5, f32=case["bias"] == "f32") if case["bias"] else None
        s["residual_t"] = normal(rows, n, f32=case["f32"]) if case["residual"] else None
        return s
    if case["op"] == "route":
        tokens, experts, fan = case["tokens"], case["experts"], case["fan"]
        # some experts are liked better than others, as a router makes them
        liked = torch.randn(experts, generator=gen, device=dev) * 0.5
        s["logits"] = (torch.randn(tokens, experts, generator=gen, device=dev) * 1.5 + liked).to(torch.float32 if case["f32"] else torch.float16)
        s["bias_t"] = -0.1 * liked if case["bias"] else None
        if case["grad"]:
            s["ids"], _ = _plain_route(s)
            s["dgates"] = normal(tokens, fan, f32=True)
        return s
    tokens, fan, n, experts = case["tokens"], case["fan"], case["n"], case["experts"]
    # the plan of the batch: routed rows sorted by expert, dropped ones last
    ids = torch.rand(tokens, experts, generator=gen, device=dev).argsort(1)[:, :fan].reshape(-1)
    ids = torch.where(torch.rand(tokens * fan, generator=gen, device=dev) < case["dropped"], experts, ids)
    order = torch.sort(ids, stable=True).indices
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(tokens * fan, device=dev)
    s["inverse"] = inverse.to(torch.int32)
    sizes = torch.bincount(ids, minlength=experts + 1)
    s["offsets"] = torch.cat([sizes.new_zeros(1), torch.cumsum(sizes, 0)])[: experts + 1].to(torch.int32)
    s["rows"] = normal(tokens * fan, n, f32=case["f32"])
    s["gates"] = torch.softmax(torch.randn(tokens, fan, generator=gen, device=dev), 1)
    if case["grad"]:
        s["dy"] = normal(tokens, n, std=0.125, f32=case["out_f32"])
    s["residual_t"] = normal(tokens, n, f32=case["out_f32"]) if case["residual"] and not case["grad"] else None
    return s


# ---- one pass ---------------------------------------------------------------

def _run_own(s):
    import dense_fp16_gemm_f16_amd as g

    if s["op"] == "fused":
        act = None if s["act"] == "none" else s["act"]
        if s["grad"]:
            dz, dbias = g.gemm_f16_fused_grad(s["dy"], s["z"], act=act, bias_grad=s["bias_grad"])
            return [t for t in (dz if act else None, dbias) if t is not None]
        out_dtype = torch.float32 if s["f32"] else torch.float16
        return g.gemm_f16_fused_nt(s["a"], s["b"], s["bias_t"], act=act, residual=s["residual_t"], return_pre=s["pre"],
                                   out_dtype=out_dtype)
    if s["op"] == "route":
        if s["grad"]:
            return g.route_grad(s["logits"], s["ids"], s["dgates"], score=s["score"], renormalize=s["renormalize"], scale=s["scale"])
        return g.route(s["logits"], s["fan"], score=s["score"], bias=s["bias_t"], groups=s["groups"], top_groups=s["top_groups"],
                       group_top=s["group_top"], renormalize=s["renormalize"], scale=s["scale"])
    if s["grad"]:
        return g.combine_rows_grad(s["dy"], s["rows"], s["inverse"], s["offsets"], s["gates"])
    return g.combine_rows(s["rows"], s["inverse"], s["offsets"], s["fan"], gates=s["gates"], residual=s["residual_t"],
                          out_dtype=torch.float32 if s["out_f32"] else torch.float16)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -(0.5 ** 0.5))
    if name == "gelu_tanh":  # 0.5 z (1 + tanh u) = z / (1 + exp(-2 u))
        return z / (1 + torch.exp(-2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p + z * p * (1 - p)
    if name == "gelu":
        return 0.5 * torch.erfc(z * -(0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    c = 2 * (2 / math.pi) ** 0.5
    p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
    return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)


def _plain_fused(s):
    if s["grad"]:
        dy = s["dy"].float()
        dz = dy if s["act"] == "none" else dy * _act_grad(s["act"], s["z"].float())
        out = [] if s["act"] == "none" else [dz.to(torch.float16)]
        return out + ([dz.sum(0, dtype=torch.float64).float()] if s["bias_grad"] else [])
    z = s["a"].float() @ s["b"].float().t()
    if s["bias_t"] is not None:
        z = z + s["bias_t"].float()
    c = _act(s["act"], z)
    if s["residual_t"] is not None:
        c = c + s["residual_t"].float()
    c = c if s["f32"] else c.to(torch.float16)
    return (c, z.to(torch.float16)) if s["pre"] else c


def _plain_route(s):
    """Scores in 64 bits: two experts a rounding apart stay in their order."""
    tokens, experts, fan, groups = s["tokens"], s["experts"], s["fan"], s["groups"]
    logits = s["logits"].double()
    if s["score"] == "softmax":
        scores = torch.exp(logits - logits.max(1, keepdim=True).values)
        scores = scores / scores.sum(1, keepdim=True)
    else:
        scores = 1 / (1 + torch.exp(-logits))
    key = logits if s["bias_t"] is None else scores + s["bias_t"].double()
    if groups > 1:
        each = (scores if s["bias_t"] is None else key).view(tokens, groups, -1)
        top = torch.sort(each, 2, descending=True).values[:, :, : s["group_top"]].sum(2)
        kept = torch.sort(top, dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        open_ = torch.zeros(tokens, groups, dtype=torch.bool, device=logits.device).scatter_(1, kept, True)
        key = torch.where(open_[:, :, None], key.view(tokens, groups, -1), -math.inf).view(tokens, experts)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :fan]
    gates = scores.gather(1, ids)
    if s["renormalize"]:
        gates = gates / gates.sum(1, keepdim=True)
    return ids.to(torch.int32), (gates * s["scale"]).float()


def _plain_route_grad(s):
    logits, ids, dg = s["logits"].float(), s["ids"].long(), s["dgates"] * s["scale"]
    if s["score"] == "softmax":
        scores = torch.exp(logits - logits.max(1, keepdim=True).values)
        scores = scores / scores.sum(1, keepdim=True)
    else:
        scores = 1 / (1 + torch.exp(-logits))
    p = scores.gather(1, ids)
    if s["renormalize"]:
        total = p.sum(1, keepdim=True)
        dp = (dg - (dg * (p / total)).sum(1, keepdim=True)) / total
    else:
        dp = dg
    picked = torch.zeros_like(scores).scatter_(1, ids, dp)
    if s["score"] == "softmax":
        dl = scores * (picked - (dp * p).sum(1, keepdim=True))
    else:
        dl = picked * scores * (1 - scores)
    return dl.to(s["logits"].dtype)


def _plain_combine(s):
    place = s["inverse"].long().view(s["tokens"], s["fan"])
    live = place < s["offsets"][-1]
    gates = torch.where(live, s["gates"], 0.0)
    if s["grad"]:
        dy = s["dy"].float()
        drows = torch.empty_like(s["rows"], dtype=torch.float16)
        drows[place.reshape(-1)] = (gates[:, :, None] * dy[:, None, :]).to(torch.float16).view(-1, s["n"])
        dgates = (s["rows"][place.reshape(-1)].float().view(s["tokens"], s["fan"], -1) * dy[:, None, :]).sum(2)
        return drows, torch.where(live, dgates, 0.0)
    y = 0.0 if s["residual_t"] is None else s["residual_t"].float()
    for f in range(s["fan"]):
        y = y + gates[:, f, None] * s["rows"][place[:, f]].float()
    return y if s["out_f32"] else y.to(torch.float16)


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "fused":
        return _plain_fused(state)
    if state["op"] == "route":
        return _plain_route_grad(state) if state["grad"] else _plain_route(state)
    return _plain_combine(state)


def work(case):
    if case["op"] == "fused":
        rows, n = case["rows"], case["n"]
        if case["grad"]:
            per = 6 if case["act"] != "none" else 2
            return {"bytes": per * rows * n + (4 * n if case["bias_grad"] else 0), "flops": 0}
        out = 4 if case["f32"] else 2
        each = out * (2 if case["residual"] else 1) + (2 if case["pre"] else 0)
        bias = {"": 0, "f16": 2, "f32": 4}[case["bias"]]
        return {"bytes": 2 * (rows + n) * case["k"] + each * rows * n + bias * n, "flops": 2 * rows * n * case["k"]}
    if case["op"] == "route":
        tokens, es = case["tokens"], 4 if case["f32"] else 2
        dense = tokens * case["experts"] * es
        return {"bytes": (2 if case["grad"] else 1) * dense + 8 * tokens * case["fan"]
                + (4 * case["experts"] if case["bias"] and not case["grad"] else 0), "flops": 0}
    tokens, fan, n = case["tokens"], case["fan"], case["n"]
    es, os_ = 4 if case["f32"] else 2, 4 if case["out_f32"] else 2
    if case["grad"]:
        return {"bytes": tokens * n * (os_ + fan * (es + 2)) + 12 * tokens * fan, "flops": 0}
    return {"bytes": tokens * n * (os_ * (2 if case["residual"] else 1) + fan * es) + 8 * tokens * fan, "flops": 0}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def _exact_fused(s):
    if s["grad"]:
        dy = s["dy"].double()
        if s["act"] == "none":
            return [dy.sum(0)]
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(_exact_act(s["act"], z), z, dy)
        return [dz, dz.sum(0)] if s["bias_grad"] else [dz]
    z = torch.mm(s["a"].double(), s["b"].double().T)
    if s["bias_t"] is not None:
        z += s["bias_t"].double()
    c = _exact_act(s["act"], z)
    if s["residual_t"] is not None:
        c = c + s["residual_t"].double()
    return (c, z) if s["pre"] else c


def _exact_gates(s, logits, ids):
    scores = torch.softmax(logits, 1) if s["score"] == "softmax" else torch.sigmoid(logits)
    p = scores.gather(1, ids)
    return s["scale"] * (p / p.sum(1, keepdim=True) if s["renormalize"] else p)


def _largest(v):
    """Index of the largest of each row, the lowest of equals."""
    at = torch.arange(v.shape[1], device=v.device)
    return torch.where(v == v.max(1, keepdim=True).values, at, v.shape[1]).min(1, keepdim=True).values


def _exact_route(s):
    logits = s["logits"].double()
    if s["grad"]:
        leaf = logits.clone().requires_grad_()
        dl, = torch.autograd.grad(_exact_gates(s, leaf, s["ids"].long()), leaf, s["dgates"].double())
        return dl
    scores = torch.softmax(logits, 1) if s["score"] == "softmax" else torch.sigmoid(logits)
    key = scores + s["bias_t"].double() if s["bias_t"] is not None else logits
    if s["groups"] > 1:
        rank = key if s["bias_t"] is not None else scores
        parts = rank.chunk(s["groups"], 1)
        value = torch.stack([p.topk(min(s["group_top"], p.shape[1]), 1).values.sum(1) for p in parts], 1)
        closed = torch.ones_like(value, dtype=torch.bool)
        for _ in range(s["top_groups"]):
            best = _largest(value.masked_fill(~closed, -math.inf))
            closed.scatter_(1, best, False)
        key = key.masked_fill(closed.repeat_interleave(s["experts"] // s["groups"], 1), -math.inf)
    picks = []
    for _ in range(s["fan"]):
        picks.append(_largest(key))
        key = key.scatter(1, picks[-1], -math.inf)
    ids = torch.cat(picks, 1)
    return ids.to(torch.int32), _exact_gates(s, logits, ids)


def _exact_combine(s):
    tokens, fan = s["tokens"], s["fan"]
    place, last = s["inverse"].long().view(tokens, fan), int(s["offsets"][-1])
    rows = s["rows"].double()
    rows[last:] = 0
    gates = s["gates"].double()
    if s["grad"]:
        dy = s["dy"].double()
        drows, dgates = torch.zeros_like(rows), torch.zeros_like(gates)
        for f in range(fan):
            drows[place[:, f]] = gates[:, f, None] * dy
            dgates[:, f] = (rows[place[:, f]] * dy).sum(1)
        drows[last:] = 0
        return drows, dgates
    y = torch.zeros(tokens, s["n"], dtype=torch.float64, device=rows.device)
    if s["residual_t"] is not None:
        y += s["residual_t"].double()
    for f in range(fan):
        y += gates[:, f, None] * rows[place[:, f]]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "fused":
        return _exact_fused(s)
    return _exact_route(s) if case["op"] == "route" else _exact_combine(s)
