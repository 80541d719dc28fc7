"""Cases of the segmented products: row grouping, the experts' products with their
gradients, and low-rank adapters beside a shared projection.

A case's ``op`` names the operator:

* ``group``  the plan of a routed batch: ids -> order, inverse, offsets
* ``nt``     experts' forward product      C_g = A_g B_g^T   (rows gathered where ``fan`` > 0)
* ``nn``     its data gradient             C_g = A_g B_g
* ``tn``     its weight gradient           C_g = A_g^T B_g
* ``lora``   y = x W^T + scale_s (x D_s^T) U_s^T, each row with its own adapter s (or none)

With ``own`` false the operators are computed in elementary torch operations in
32 bits, rounded once at the end; with it true by the library.
"""
import math

import torch

own = False


# ---- the cases --------------------------------------------------------------

def listed():
    return [
        # a decoding step of 64 sequences, two experts each: the plan before every routed layer
        {"name": "plan of a decode batch", "op": "group", "rows": 128, "groups": 8, "empty": 0},
        # a training batch of 16384 tokens, eight of 64 experts each
        {"name": "plan of a training batch", "op": "group", "rows": 131072, "groups": 64, "empty": 3},
        # eight sequences decode one token each: the weights of all the experts are read for 16 rows
        {"name": "experts, decode", "op": "nt", "rows": 16, "groups": 8, "empty": 0, "n": 4096, "k": 2048, "fan": 2, "f32": False},
        # 8192 tokens, two of eight experts each: a training forward pass or a long prompt
        {"name": "experts, forward", "op": "nt", "rows": 16384, "groups": 8, "empty": 0, "n": 4096, "k": 2048, "fan": 2, "f32": False},
        # ragged: no size a multiple of a tile, three experts without a row
        {"name": "experts, ragged", "op": "nt", "rows": 5000, "groups": 13, "empty": 3, "n": 3000, "k": 1000, "fan": 0, "f32": False},
        # the training step's gradient of the experts' inputs
        {"name": "data gradient", "op": "nn", "rows": 16384, "groups": 8, "empty": 0, "n": 2048, "k": 4096, "f32": False},
        {"name": "data gradient, ragged", "op": "nn", "rows": 5000, "groups": 13, "empty": 3, "n": 1000, "k": 3000, "f32": True},
        # the training step's gradient of the experts' weights, in fp32 for the optimizer
        {"name": "weight gradient", "op": "tn", "rows": 16384, "groups": 8, "empty": 0, "n": 2048, "k": 4096, "f32": True},
        {"name": "weight gradient, ragged", "op": "tn", "rows": 5000, "groups": 13, "empty": 3, "n": 1000, "k": 3000, "f32": False},
        # one request decodes: the latency of a projection
        {"name": "adapters, one token", "op": "lora", "rows": 1, "adapters": 4, "rank": 16, "n": 4096, "k": 4096, "runs": False},
        # 48 requests decode together with up to 32 different adapters
        {"name": "adapters, decode", "op": "lora", "rows": 48, "adapters": 32, "rank": 16, "n": 4096, "k": 4096, "runs": False},
        # prompts of several requests, one after the other
        {"name": "adapters, prompts", "op": "lora", "rows": 4096, "adapters": 8, "rank": 64, "n": 4096, "k": 4096, "runs": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A matrix width: mostly whole 16-byte chunks, one in five any size."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.2 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["group", "nt", "nt", "nn", "tn", "lora", "lora"])
    if op == "group":
        groups = _log(rng, 1, 256)
        return {"op": op, "rows": _log(rng, 1, 131072), "groups": groups, "empty": rng.randrange(0, (groups + 1) // 2)}
    if op == "lora":
        return {"op": op, "rows": _log(rng, 1, 4096), "adapters": _log(rng, 1, 64), "rank": rng.choice([4, 8, 12, 16, 16, 24, 32, 64]),
                "n": _width(rng, 128, 4096), "k": _width(rng, 128, 4096), "runs": rng.random() < 0.5}
    groups = _log(rng, 1, 64)
    n = _width(rng, 64, 4096)
    k = _width(rng, 64, 4096)
    while groups * n * k > 8 * 4096 * 2048:  # no dearer than the largest listed case
        groups = max(1, groups // 2)
        n, k = (n, max(8, k // 16 * 8)) if k > n else (max(8, n // 16 * 8), k)
    rows = min(_log(rng, 1, 16384), 16384 * 4096 * 2048 // (n * k))
    case = {"op": op, "rows": rows, "groups": groups, "empty": rng.randrange(0, (groups + 1) // 2), "n": n, "k": k,
            "f32": rng.random() < 0.5}
    if op == "nt":
        case["fan"] = rng.choice([0, 1, 2, 4])
    return case


# ---- inputs -----------------------------------------------------------------

def _route(rows, groups, empty, gen):
    """Group of each row: uneven as a router makes them, `empty` groups without a row, the others with one at least where the rows suffice."""
    dev = gen.device
    used = torch.randperm(groups, generator=gen, device=dev)[: groups - empty]
    share = torch.softmax(torch.randn(len(used), generator=gen, device=dev), 0)
    edge = torch.cumsum(share, 0)
    pick = torch.searchsorted(edge, torch.rand(rows, generator=gen, device=dev)).clamp(max=len(used) - 1)
    pick[: min(rows, len(used))] = torch.arange(min(rows, len(used)), device=dev)
    return used[pick[torch.randperm(rows, generator=gen, device=dev)]].to(torch.int32)


def _plan(ids, groups):
    key = torch.where((ids >= 0) & (ids < groups), ids, groups).long()
    sizes = torch.bincount(key, minlength=groups + 1)
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    offsets = torch.cat([sizes.new_zeros(1), torch.cumsum(sizes, 0)])[: groups + 1].to(torch.int32)
    return order, offsets, sizes[:groups].tolist()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.float16)

    s = dict(case)
    rows = case["rows"]
    if case["op"] == "group":
        s["ids"] = _route(rows, case["groups"], case["empty"], gen)
        return s
    n, k = case["n"], case["k"]
    if case["op"] == "lora":
        adapters, rank = case["adapters"], case["rank"]
        if case["runs"]:  # prompts: each request's rows together
            cuts = torch.rand(adapters - 1, generator=gen, device=dev).sort().values if adapters > 1 else torch.zeros(0, device=dev)
            at = (torch.arange(rows, device=dev) + 0.5) / rows
            owner = torch.randperm(adapters, generator=gen, device=dev)
            s["ids"] = owner[torch.searchsorted(cuts, at)].to(torch.int32)
        else:  # decoding: any adapter, and one request in eight without one
            ids = torch.randint(0, adapters, (rows,), generator=gen, device=dev)
            s["ids"] = torch.where(torch.rand(rows, generator=gen, device=dev) < 0.125, -1, ids).to(torch.int32)
        s["x"] = normal(rows, k)
        s["w"] = normal(n, k, std=k ** -0.5)
        s["down"] = normal(adapters, rank, k, std=k ** -0.5)
        s["up"] = normal(adapters, n, rank, std=rank ** -0.5)
        s["scale"] = torch.rand(adapters, generator=gen, device=dev) + 0.5
        s["order"], s["offsets"], _ = _plan(s["ids"], adapters)
        return s
    groups = case["groups"]
    ids = _route(rows, groups, case["empty"], gen)
    order, s["offsets"], s["sizes"] = _plan(ids, groups)
    if case["op"] == "nt":
        fan = case["fan"]
        s["index"] = order if fan else None
        s["a"] = normal(-(-rows // fan) if fan else rows, k)
        s["b"] = normal(groups, n, k, std=k ** -0.5)
    elif case["op"] == "nn":
        s["a"] = normal(rows, k, std=0.125)
        s["b"] = normal(groups, k, n, std=k ** -0.5)
    else:
        s["a"] = normal(rows, k, std=0.125)
        s["b"] = normal(rows, n)
    return s


# ---- one pass ---------------------------------------------------------------

def _run_own(s):
    import dense_fp16_gemm_f16_amd as g

    op = s["op"]
    if op == "group":
        return tuple(g.group_rows(s["ids"], s["groups"]))
    if op == "lora":
        return g.gemm_f16_lora_nt(s["x"], s["w"], s["down"], s["up"], s["ids"], s["order"], s["offsets"], s["scale"])
    out_dtype = torch.float32 if s["f32"] else torch.float16
    if op == "nt":
        return g.gemm_f16_grouped_nt(s["a"], s["b"], s["offsets"], index=s["index"], fan=s["fan"] or 1, out_dtype=out_dtype)
    if op == "nn":
        return g.gemm_f16_grouped_nn(s["a"], s["b"], s["offsets"], out_dtype=out_dtype)
    return g.gemm_f16_grouped_tn(s["a"], s["b"], s["offsets"], out_dtype=out_dtype)


def _plain_group(ids, groups):
    key = torch.where((ids >= 0) & (ids < groups), ids, groups)
    order = torch.sort(key, stable=True).indices
    inverse = torch.empty_like(order)
    inverse[order] = torch.arange(len(ids), device=ids.device)
    edges = torch.arange(groups + 1, device=ids.device, dtype=key.dtype)
    offsets = (key[None, :] < edges[:, None]).sum(1)
    return order.to(torch.int32), inverse.to(torch.int32), offsets.to(torch.int32)


def _plain_lora(s):
    adapters, rank, k = s["down"].shape
    x = s["x"].float()
    h = (x @ s["down"].reshape(adapters * rank, k).float().t()).view(-1, adapters, rank)
    mine = s["ids"][:, None] == torch.arange(adapters, device=x.device)
    h = torch.where(mine[:, :, None], h * s["scale"][None, :, None], 0.0)
    up = s["up"].float().permute(0, 2, 1).reshape(adapters * rank, -1)
    y = x @ s["w"].float().t() + h.reshape(len(x), -1) @ up
    return y.to(torch.float16)


def run(state):
    if own:
        return _run_own(state)
    s = state
    if s["op"] == "group":
        return _plain_group(s["ids"], s["groups"])
    if s["op"] == "lora":
        return _plain_lora(s)
    a = s["a"]
    if s["op"] == "nt" and s["index"] is not None:
        a = a[s["index"].long() // s["fan"]]
    parts = torch.split(a.float(), s["sizes"])
    if s["op"] == "nt":
        out = torch.cat([p @ w.t() for p, w in zip(parts, s["b"].float())])
    elif s["op"] == "nn":
        out = torch.cat([p @ w for p, w in zip(parts, s["b"].float())])
    else:
        out = torch.stack([p.t() @ q for p, q in zip(parts, torch.split(s["b"].float(), s["sizes"]))])
    return out if s["f32"] else out.to(torch.float16)


def work(case):
    rows = case["rows"]
    if case["op"] == "group":
        return {"bytes": 4 * (3 * rows + case["groups"] + 1), "flops": 0}
    n, k = case["n"], case["k"]
    if case["op"] == "lora":
        used = min(case["adapters"], rows)
        low = case["rank"] * (n + k)
        return {"bytes": 2 * (rows * k + n * k + used * low + rows * n), "flops": 2 * rows * (n * k + low)}
    size = 4 if case["f32"] else 2
    used = min(case["groups"] - case["empty"], rows)
    if case["op"] == "tn":
        moved = 2 * rows * (n + k) + size * case["groups"] * n * k
    elif case["op"] == "nt" and case["fan"]:
        moved = 2 * (-(-rows // case["fan"]) * k + used * n * k) + size * rows * n + 4 * rows
    else:
        moved = 2 * (rows * k + used * n * k) + size * rows * n
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ---- the definition in 64 bits ----------------------------------------------

def exact(case, seed):
    if case["op"] == "group":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "lora":
        x = s["x"].double()
        y = torch.mm(x, s["w"].double().T)
        for i in range(case["adapters"]):
            rows = (s["ids"] == i).nonzero().flatten()
            low = torch.mm(x[rows], s["down"][i].double().T) * s["scale"][i].double()
            y[rows] += torch.mm(low, s["up"][i].double().T)
        return y
    edges = s["offsets"].tolist()
    a, b = s["a"].double(), s["b"]
    if case["op"] == "tn":
        out = torch.zeros(case["groups"], case["k"], case["n"], dtype=torch.float64, device=a.device)
        for i in range(case["groups"]):
            out[i] = torch.mm(a[edges[i]:edges[i + 1]].T, b[edges[i]:edges[i + 1]].double())
        return out
    if case["op"] == "nt" and case["fan"]:
        a = a[torch.div(s["index"].long(), case["fan"], rounding_mode="floor")]
    out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=a.device)
    for i in range(case["groups"]):
        w = b[i].double()
        out[edges[i]:edges[i + 1]] = torch.mm(a[edges[i]:edges[i + 1]], w.T if case["op"] == "nt" else w)
    return out
