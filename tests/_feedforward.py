"""Plain 64-bit definitions of the feed-forward layer's operators, and the
bounds the GPU results are held to (test infrastructure).

Bounds, u = 2^-24 (half a step of fp32):

* z = sum + bias: k + 1 terms in fp32, in any order and with truncating adders,
  off by at most (k + 2) 2u times the sum of their magnitudes.
* An activation passes that on by at most its steepest slope (1.13), and adds
  its own roundings, relative to its value: the hardware's exp2 and rcp are good
  to one step (2u), every other operation to u, and exp(x) computed as exp2 of
  a rounded product is off by |x| u more for each rounding of x.
    silu:      (|z| + 6) 2u
    gelu_tanh: w has six roundings, constants included: (6 |w| + 8) u
    gelu:      the fitted tail 4.8e-7 and a reciprocal's step, below 2^-20;
               exp(-z^2/2): two roundings: (z^2 2 u / 2 + ..) <= z^2 2^-22
* The last rounding: half a step of the output's type.
"""
import math

import torch

from tests import _segments as seg

U = 2.0**-24
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]
SLOPE = 1.13


def _w(z):
    return math.sqrt(8 / math.pi) * (z + 0.044715 * z**3)


def cdf(z):
    """The normal distribution; torch.special.ndtr computes 1 + erf, which loses the lower tail."""
    return 0.5 * torch.erfc(z * -(0.5**0.5))


def act(name, z):
    if name is None:
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * cdf(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(_w(z))
    return z * torch.sigmoid(z)


def act_error(name, z):
    """Bound on an activation's own error, relative to its value."""
    if name == "gelu":
        return z**2 * 2.0**-22 + 2.0**-20
    if name == "gelu_tanh":
        return (6 * _w(z).abs() + 8) * U
    if name == "silu":
        return (z.abs() + 6) * 2 * U
    return torch.zeros_like(z)


def fused(a, b, bias, name, residual):
    """(c, z, bound on c before its rounding, bound on z) in float64."""
    a, b = a.double(), b.double()
    z = torch.mm(a, b.T.contiguous())
    mag = torch.mm(a.abs(), b.abs().T.contiguous())
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ez = (a.shape[1] + 2) * 2 * U * mag
    y = act(name, z)
    err = ez * (SLOPE if name else 1.0) + act_error(name, z) * (y.abs() + ez)
    if residual is not None:
        r = residual.double()
        err = err + 2 * U * (y.abs() + r.abs())
        y = y + r
    return y, z, err, ez


def act_grad(name, z):
    if name is None:
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return cdf(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        s = torch.sigmoid(_w(z))
        return s + z * s * torch.sigmoid(-_w(z)) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s + z * s * torch.sigmoid(-z)


def act_grad_error(name, z):
    """Bound on the error of act'(z): both terms' roundings, and for z > 0 that of 1 - s
    against 1 (u, and s's own error, 2u, of which it is the difference)."""
    if name in (None, "relu"):
        return torch.zeros_like(z)
    if name == "gelu":
        tail = cdf(z) + z.abs() * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return (z**2 * 2.0**-22 + 2.0**-20) * tail + U
    slope = math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z) if name == "gelu_tanh" else torch.ones_like(z)
    w = _w(z) if name == "gelu_tanh" else z
    s = torch.sigmoid(w)
    m = s + z.abs() * slope * s * torch.sigmoid(-w)
    return (6 * w.abs() + 16) * 2 * U * m + torch.where(z > 0, 4 * U * z.abs() * slope, 0.0)


def fused_grad(dy, pre, name):
    """(dz, dbias, bound on dz before its rounding, bound on dbias) in float64."""
    dy = dy.double()
    z = dy if pre is None else pre.double()
    g = act_grad(name, z)
    dz = dy * g
    err = dy.abs() * act_grad_error(name, z) + U * dz.abs()
    return dz, dz.sum(0), err, err.sum(0) + dz.shape[0] * 2 * U * dz.abs().sum(0)


def route(logits, fan, score="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    """(ids, gates) in float64, an expert at a time, on the CPU."""
    l = logits.double().cpu()
    tokens, experts = l.shape
    none = torch.isnan(l) | (l == -math.inf)
    l = torch.where(none, -math.inf, l)
    if score == "softmax":
        m = l.max(1, keepdim=True).values
        e = torch.where(l == m, 1.0, torch.exp(l - torch.where(torch.isinf(m), 0.0, m)))
        e = torch.where(torch.isinf(m) & (l != m), 0.0, e)
        e = torch.where(none, 0.0, e)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = torch.where(none, 0.0, torch.sigmoid(l))
    key = l.clone() if bias is None else s + bias.double().cpu()
    key = torch.where(none | torch.isnan(key), -math.inf, key)
    value = torch.where(none, -math.inf, s) if bias is None and group_top == 2 else key
    per = experts // groups
    ids = torch.full((tokens, fan), -1, dtype=torch.int64)
    gates = torch.zeros(tokens, fan, dtype=torch.float64)
    for t in range(tokens):
        open_ = list(range(groups))
        if groups > 1:
            worth = []
            for g in range(groups):
                v = sorted(value[t, g * per:(g + 1) * per].tolist(), reverse=True)[:group_top]
                v = [x for x in v if x != -math.inf]
                worth.append(sum(v) if v else -math.inf)
            order = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            open_ = [g for g in order if worth[g] != -math.inf]
        able = [e for g in open_ for e in range(g * per, (g + 1) * per) if key[t, e] != -math.inf]
        chosen = sorted(able, key=lambda e: (-float(key[t, e]), e))[:fan]
        if not chosen:
            continue
        if renormalize:  # scores without a common factor: the same, where they underflow too
            x = torch.tensor([float(l[t, e]) for e in chosen], dtype=torch.float64)
            p = x if score == "softmax" else x.clamp(max=0)  # sigmoid(x) = exp(min(x, 0)) / (1 + exp(-|x|))
            top = p.max()
            p = torch.where(p == top, 1.0, torch.exp(torch.where(p == top, 0.0, p - top)))
            p = p if score == "softmax" else p / (1 + torch.exp(-x.abs()))
            p = p / p.sum()
        else:
            p = s[t, chosen]
        ids[t, :len(chosen)] = torch.tensor(chosen)
        gates[t, :len(chosen)] = scale * p
    return ids, gates


def gates_of(logits, ids, score, renormalize, scale):
    """The gates as a differentiable function of float64 logits, the choice fixed (-1: none)."""
    live = ids >= 0
    at = ids.clamp(min=0)
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    p = torch.where(live, s.gather(1, at), 0.0)
    return scale * (p / p.sum(1, keepdim=True) if renormalize else p)


def combine(rows, inverse, last, fan, gates, residual):
    """(y, bound before its rounding) in float64."""
    place = inverse.long().view(-1, fan)
    live = place < last
    r = torch.where(live.reshape(-1)[:, None], rows.double()[place.reshape(-1)], 0.0).view(len(place), fan, -1)
    w = torch.ones(len(place), fan, dtype=torch.float64, device=rows.device) if gates is None else gates.double()
    each = r * w[:, :, None]
    y, mag = each.sum(1), each.abs().sum(1)
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, (fan + 1) * 2 * U * mag


def combine_grad(dy, rows, inverse, last, gates):
    """(drows, dgates, bound on drows before its rounding, bound on dgates) in float64."""
    tokens, fan = gates.shape
    place = inverse.long().view(tokens, fan)
    live = (place < last)
    d = dy.double()
    drows = torch.zeros(tokens * fan, dy.shape[1], dtype=torch.float64, device=dy.device)
    g = torch.where(live, gates.double(), 0.0)
    drows[place.reshape(-1)] = (g[:, :, None] * d[:, None, :]).reshape(tokens * fan, -1)
    r = torch.where(live.reshape(-1)[:, None], rows.double()[place.reshape(-1)], 0.0).view(tokens, fan, -1)
    each = r * d[:, None, :]
    return drows, each.sum(2), U * drows.abs(), (dy.shape[1] + 1) * 2 * U * each.abs().sum(2)


worst, eighths, normal = seg.worst, seg.eighths, seg.normal
