"""Segmented products: matrix products whose rows fall into groups of sizes
that only the GPU knows (the tokens of each expert, the requests of each
adapter).

* ``group_rows``           ids -> (order, inverse, offsets)
* ``gemm_f16_grouped_nt``  experts' forward product, C_g = A_g B_g^T
* ``gemm_f16_grouped_nn``  its gradient by the rows, C_g = A_g B_g
* ``gemm_f16_grouped_tn``  its gradient by the weights, C_g = A_g^T B_g
* ``gemm_f16_lora_nt``     X W^T and each row's own low-rank adapter

Every call is asynchronous on ``stream`` (default: torch's current stream),
never waits for the GPU and captures into HIP graphs.  Outputs and the
workspace are allocated on that stream.  The arguments' contracts are those of
``include/gemm_f16.h``; shapes, types and devices are checked here, and a
status of the library raises ``GemmError``.
"""
from __future__ import annotations

import contextlib

import dense_fp16_gemm_f16_amd as _g

GROUPED_NT = 0
GROUPED_NN = 1
GROUPED_TN = 2

_ON = contextlib.nullcontext()


def _operand(name, t, dtype, shape, device):
    """t is a contiguous tensor of dtype on device; a None in shape takes any size."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be on the same GPU as the other operands")
    if len(t.shape) != len(shape) or any(w is not None and w != v for v, w in zip(t.shape, shape)):
        raise ValueError(f"{name}: expected shape {tuple('any' if w is None else w for w in shape)}, "
                         f"got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def _on(device, stream):
    """(context, stream handle): allocations inside the context belong to the stream."""
    import torch

    if stream is None:
        handle = torch.cuda.current_stream(device).cuda_stream
        return (_ON if torch.cuda.current_device() == device.index else torch.cuda.device(device)), handle
    return torch.cuda.stream(stream), stream.cuda_stream


def _out(out, shape, dtype, device):
    import torch

    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _operand("out", out, dtype, shape, device)
    return out


def _workspace(size, device):
    import torch

    if size < 0:
        raise _g.GemmError(size)
    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def _ptr(t):
    return None if t is None else (t.data_ptr() or None)


def _check(rc):
    if rc != _g.OK:
        raise _g.GemmError(rc)


def group_rows(ids, groups: int, *, stream=None):
    """The plan of a routed batch: (order, inverse, offsets), all int32.

    ``ids`` (int32 or int64, any shape, contiguous) gives the group of each
    row, rows counted through the flattened ids: with ids [tokens, fan], row r
    is token r // fan.  ``order`` lists the rows sorted by group, rows of one
    group in their order; ``inverse`` is the place of each row in it;
    ``offsets`` [groups+1] holds each group's first place.  Ids outside
    [0, groups) belong to no group: their rows come last, from offsets[-1] on.
    """
    import torch

    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64")
    if not ids.is_cuda:
        raise ValueError("ids must be on a GPU")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")
    L, rows, device = _g.lib(), ids.numel(), ids.device
    context, handle = _on(device, stream)
    with context:
        ws = _workspace(L.gemm_f16_group_rows_workspace(rows, groups), device)
        order = torch.empty(rows, dtype=torch.int32, device=device)
        inverse = torch.empty(rows, dtype=torch.int32, device=device)
        offsets = torch.empty(groups + 1, dtype=torch.int32, device=device)
        _check(L.gemm_f16_group_rows(rows, groups, _ptr(ids), ids.element_size(), _ptr(order), _ptr(inverse),
                                     _ptr(offsets), _ptr(ws), ws.numel() if ws is not None else 0, handle or None))
    return order, inverse, offsets


def _grouped(kind, a, b, offsets, index, fan, out_dtype, out, stream):
    import torch

    if a.dim() != 2 or b.dim() != (2 if kind == GROUPED_TN else 3):
        raise ValueError("expected a [rows,K] and b [rows,N]" if kind == GROUPED_TN
                         else "expected a [rows,K] and b of three dimensions")
    if out_dtype not in (torch.float16, torch.float32):
        raise TypeError("out_dtype must be float16 or float32")
    device = a.device
    a_rows, k = a.shape
    rows = a_rows if index is None else index.numel()
    _operand("a", a, torch.float16, (None, None), device)
    if kind == GROUPED_NT:
        _operand("b", b, torch.float16, (None, None, k), device)
    elif kind == GROUPED_NN:
        _operand("b", b, torch.float16, (None, k, None), device)
    else:
        _operand("b", b, torch.float16, (a_rows, None), device)
    groups = offsets.numel() - 1 if kind == GROUPED_TN else b.shape[0]
    n = b.shape[1] if kind != GROUPED_NN else b.shape[2]
    _operand("offsets", offsets, torch.int32, (groups + 1,), device)
    if index is not None:
        _operand("index", index, torch.int32, (rows,), device)
    L = _g.lib()
    size = L.gemm_f16_grouped_workspace(kind, rows, groups, n, k)
    context, handle = _on(device, stream)
    with context:
        ws = _workspace(size, device)
        out = _out(out, (groups, k, n) if kind == GROUPED_TN else (rows, n), out_dtype, device)
        f32 = int(out_dtype == torch.float32)
        if kind == GROUPED_NT:
            rc = L.gemm_f16_grouped_nt(rows, groups, n, k, _ptr(a), a_rows, _ptr(b), _ptr(offsets), _ptr(index), fan,
                                       _ptr(out), f32, _ptr(ws), size, handle or None)
        else:
            call = L.gemm_f16_grouped_nn if kind == GROUPED_NN else L.gemm_f16_grouped_tn
            rc = call(rows, groups, n, k, _ptr(a), _ptr(b), _ptr(offsets), _ptr(out), f32, _ptr(ws), size,
                      handle or None)
        _check(rc)
    return out


def _f16(dtype):
    import torch

    return torch.float16 if dtype is None else dtype


def gemm_f16_grouped_nt(a, b, offsets, *, index=None, fan: int = 1, out_dtype=None, out=None, stream=None):
    """out[r] = a[index[r] // fan] @ b[g].T for each row r of segment g.

    a float16 [tokens,K], b float16 [groups,N,K], offsets int32 [groups+1];
    without ``index`` row r takes a[r].  With (order, _, offsets) =
    group_rows(ids, groups) of ids [tokens, fan], ``index=order, fan=fan``
    gathers each routed row's token.  ``out_dtype`` float16 (default) or
    float32; rows behind offsets[-1] are zeros.
    """
    return _grouped(GROUPED_NT, a, b, offsets, index, fan, _f16(out_dtype), out, stream)


def gemm_f16_grouped_nn(a, b, offsets, *, out_dtype=None, out=None, stream=None):
    """out[r] = a[r] @ b[g] for each row r of segment g: a float16 [rows,K],
    b float16 [groups,K,N].  With a the gradient of gemm_f16_grouped_nt's
    output and b its weights, the gradient of its rows."""
    return _grouped(GROUPED_NN, a, b, offsets, None, 1, _f16(out_dtype), out, stream)


def gemm_f16_grouped_tn(a, b, offsets, *, out_dtype=None, out=None, stream=None):
    """out[g] = a[rows of g].T @ b[rows of g]: a float16 [rows,K], b float16
    [rows,N], out [groups,K,N], zeros for an empty segment.  With a the
    gradient of gemm_f16_grouped_nt's output and b its rows, the gradient of
    its weights."""
    return _grouped(GROUPED_TN, a, b, offsets, None, 1, _f16(out_dtype), out, stream)


def gemm_f16_lora_nt(x, w, down, up, ids, order, offsets, scale=None, *, out=None, stream=None):
    """y[r] = x[r] @ w.T + scale[s] * (x[r] @ down[s].T) @ up[s].T, s = ids[r].

    x float16 [rows,K], w float16 [N,K], down float16 [adapters,rank,K], up
    float16 [adapters,N,rank], ids int32 [rows] (outside [0, adapters): no
    adapter), (order, _, offsets) = group_rows(ids, adapters), scale float32
    [adapters] (default: ones).  Returns float16 [rows,N].
    """
    import torch

    if x.dim() != 2 or w.dim() != 2 or down.dim() != 3:
        raise ValueError("expected x [rows,K], w [N,K] and down [adapters,rank,K]")
    device = x.device
    rows, k = x.shape
    n = w.shape[0]
    adapters, rank = down.shape[:2]
    _operand("x", x, torch.float16, (None, None), device)
    _operand("w", w, torch.float16, (None, k), device)
    _operand("down", down, torch.float16, (None, None, k), device)
    _operand("up", up, torch.float16, (adapters, n, rank), device)
    _operand("ids", ids, torch.int32, (rows,), device)
    _operand("order", order, torch.int32, (rows,), device)
    _operand("offsets", offsets, torch.int32, (adapters + 1,), device)
    if scale is not None:
        _operand("scale", scale, torch.float32, (adapters,), device)
    L = _g.lib()
    size = L.gemm_f16_lora_workspace(rows, n, k, adapters, rank)
    context, handle = _on(device, stream)
    with context:
        ws = _workspace(size, device)
        out = _out(out, (rows, n), torch.float16, device)
        _check(L.gemm_f16_lora_nt(rows, n, k, adapters, rank, _ptr(x), _ptr(w), _ptr(down), _ptr(up), _ptr(ids),
                                  _ptr(order), _ptr(offsets), _ptr(scale), _ptr(out), _ptr(ws), size, handle or None))
    return out
