"""Plain 64-bit definitions of the segmented products, and the bounds the
GPU results are held to (test infrastructure).

The bound of a product: fp16 products are exact in fp32, and a sum of t terms
in fp32, in any order and with truncating adders, is off by at most
t 2^-23 times the sum of their magnitudes; one rounding to fp16 adds half a
step, 2^-11 of the value or 2^-25 below the normal range.  Inputs that are
multiples of 1/8 up to 1 have exact sums (below 2^18 steps of 1/64 for up to
4096 terms), so their results have one right answer.
"""
import numpy as np
import torch

EPS = {torch.float16: 2.0**-11, torch.float32: 0.0}
TINY = {torch.float16: 2.0**-25, torch.float32: 0.0}


def group_rows(ids, groups):
    ids = np.asarray(ids, dtype=np.int64).reshape(-1)
    key = np.where((ids >= 0) & (ids < groups), ids, groups)
    order = np.argsort(key, kind="stable")
    inverse = np.empty_like(order)
    inverse[order] = np.arange(len(ids))
    offsets = np.searchsorted(key[order], np.arange(groups + 1), side="left")
    return order.astype(np.int32), inverse.astype(np.int32), offsets.astype(np.int32)


def grouped(kind, a, b, offsets, index=None, fan=1):
    """(result, sum of magnitudes, terms of a sum) in float64 on the tensors' device."""
    off = [int(v) for v in offsets]
    groups = len(off) - 1
    a, b = a.double(), b.double()
    if index is not None:
        a = a[torch.div(index.long(), fan, rounding_mode="floor")]
    if kind == "tn":
        k, n = a.shape[1], b.shape[1]
        c = torch.zeros(groups, k, n, dtype=torch.float64, device=a.device)
        s = torch.zeros_like(c)
        for g in range(groups):
            x, y = a[off[g]:off[g + 1]], b[off[g]:off[g + 1]]
            c[g], s[g] = torch.mm(x.T, y), torch.mm(x.abs().T, y.abs())
        return c, s, max([off[g + 1] - off[g] for g in range(groups)] + [1])
    n = b.shape[1] if kind == "nt" else b.shape[2]
    c = torch.zeros(a.shape[0], n, dtype=torch.float64, device=a.device)
    s = torch.zeros_like(c)
    for g in range(groups):
        x = a[off[g]:off[g + 1]]
        w = b[g].T.contiguous() if kind == "nt" else b[g]
        c[off[g]:off[g + 1]], s[off[g]:off[g + 1]] = torch.mm(x, w), torch.mm(x.abs(), w.abs())
    return c, s, max(1, a.shape[1])


def lora(x, w, down, up, ids, scale):
    """(result, bound on the error before the last rounding) in float64."""
    x, w, down, up = x.double(), w.double(), down.double(), up.double()
    k, rank = x.shape[1], down.shape[1]
    y = torch.mm(x, w.T.contiguous())
    # the terms of both products are summed in one fp32 accumulator
    err = torch.mm(x.abs(), w.abs().T.contiguous())
    for s in range(down.shape[0]):
        rows = (ids == s).nonzero().flatten()
        f = 1.0 if scale is None else float(scale[s])
        low = torch.mm(x[rows], down[s].T.contiguous()) * f
        mag = torch.mm(x[rows].abs(), down[s].abs().T.contiguous()) * abs(f)
        y[rows] += torch.mm(low, up[s].T.contiguous())
        err[rows] += torch.mm(mag, up[s].abs().T.contiguous())
    # h: k terms and its scale; its two bf16 parts without the least product (2^-17); then
    # k + 3 rank terms
    return y, err * ((2 * k + 3 * rank + 4) * 2.0**-23 + 2.0**-17)


def worst(got, ref, err, dtype):
    """Largest error over its bound; the bound err of the sum before the last rounding."""
    tol = err * (1 + EPS[dtype]) + EPS[dtype] * ref.abs() + TINY[dtype] + 1e-300
    off = (got.double() - ref).abs()
    assert bool(torch.isfinite(off).all()), "a result is not finite"
    return float((off / tol).max()) if off.numel() else 0.0


def offsets_of(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32)


def eighths(gen, *shape):
    return (torch.randint(-8, 9, shape, generator=gen, device=gen.device) / 8.0).to(torch.float16)


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=gen.device) * std).to(torch.float16)
