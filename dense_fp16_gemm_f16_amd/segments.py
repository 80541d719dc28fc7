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
workspace are allocated on that stream; for operands of another one the caller
orders the streams and keeps the tensors (``record_stream``).  The arguments' contracts are those of
``include/gemm_f16.h``; shapes, types and devices are checked here, and a
status of the library raises ``GemmError``.
"""
from __future__ import annotations

import functools

import dense_fp16_gemm_f16_amd as _g


def _operand(name, t, dtype, shape, device):
    """t must be a contiguous tensor of this dtype and shape on this GPU."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on the same GPU as the other operands")
    raise ValueError(f"{name} must be contiguous (row-major)")


def _first(name, t, dtype):
    """The device of a call: that of its first operand, which must be on a GPU."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    return t.device


def _launch(device, stream, call):
    """call(stream handle) with that stream current, so that what it allocates
    belongs to the stream."""
    import torch

    if stream is not None:
        if stream.device != device:  # kernels run where the stream is
            raise ValueError("stream must be on the same GPU as the operands")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    index = device.index
    if torch._C._cuda_getDevice() == index:
        return call(torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(device):
        return call(torch._C._cuda_getCurrentRawStream(index))


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name, *sizes):
    size = getattr(_g.lib(), name)(*sizes)
    if size < 0:
        raise _g.GemmError(size)
    return size


def _result(out, shape, dtype, device):
    import torch

    if out is None:
        return torch.empty(*shape, dtype=dtype, device=device)  # (as a tuple the sizes take 0.4 us longer)
    _operand("out", out, dtype, shape, device)
    return out


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

    if ids.dtype is not torch.int32 and ids.dtype is not torch.int64:
        raise TypeError("ids must be int32 or int64")
    device, rows = _first("ids", ids, ids.dtype), ids.numel()
    size = _workspace_bytes("gemm_f16_group_rows_workspace", rows, groups)

    def call(handle):
        order = torch.empty(rows, dtype=torch.int32, device=device)
        inverse = torch.empty(rows, dtype=torch.int32, device=device)
        offsets = torch.empty(groups + 1, dtype=torch.int32, device=device)
        ws = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        rc = _g.lib().gemm_f16_group_rows(
            rows, groups, ids.data_ptr(), ids.element_size(), order.data_ptr(), inverse.data_ptr(),
            offsets.data_ptr(), ws.data_ptr() if size else None, size, handle)
        if rc:
            raise _g.GemmError(rc)
        return order, inverse, offsets

    return _launch(device, stream, call)


def _out_type(out_dtype):
    import torch

    if out_dtype is None:
        return torch.float16
    if out_dtype is not torch.float16 and out_dtype is not torch.float32:
        raise TypeError("out_dtype must be float16 or float32")
    return out_dtype


def gemm_f16_grouped_nt(a, b, offsets, *, index=None, fan: int = 1, out_dtype=None, out=None, stream=None):
    """out[r] = a[index[r] // fan] @ b[g].T for each row r of segment g.

    a float16 [tokens,K], b float16 [groups,N,K], offsets int32 [groups+1];
    without ``index`` row r takes a[r].  With (order, _, offsets) =
    group_rows(ids, groups) of ids [tokens, fan], ``index=order, fan=fan``
    gathers each routed row's token.  ``out_dtype`` float16 (default) or
    float32; rows behind offsets[-1] are zeros.
    """
    import torch

    dtype = _out_type(out_dtype)
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("expected a [rows,K] and b [groups,N,K]")
    device = _first("a", a, torch.float16)
    (a_rows, k), (groups, n, _) = a.shape, b.shape
    rows = a_rows if index is None else index.numel()
    _operand("b", b, torch.float16, (groups, n, k), device)
    _operand("offsets", offsets, torch.int32, (groups + 1,), device)
    if index is not None:
        _operand("index", index, torch.int32, (rows,), device)

    def call(handle):
        c = _result(out, (rows, n), dtype, device)
        rc = _g.lib().gemm_f16_grouped_nt(
            rows, groups, n, k, a.data_ptr(), a_rows, b.data_ptr(), offsets.data_ptr(),
            None if index is None else index.data_ptr(), fan, c.data_ptr(), dtype is torch.float32, handle)
        if rc:
            raise _g.GemmError(rc)
        return c

    return _launch(device, stream, call)


def gemm_f16_grouped_nn(a, b, offsets, *, out_dtype=None, out=None, stream=None):
    """out[r] = a[r] @ b[g] for each row r of segment g: a float16 [rows,K],
    b float16 [groups,K,N].  With a the gradient of gemm_f16_grouped_nt's
    output and b its weights, the gradient of its rows."""
    import torch

    dtype = _out_type(out_dtype)
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("expected a [rows,K] and b [groups,K,N]")
    device = _first("a", a, torch.float16)
    (rows, k), (groups, _, n) = a.shape, b.shape
    _operand("b", b, torch.float16, (groups, k, n), device)
    _operand("offsets", offsets, torch.int32, (groups + 1,), device)

    def call(handle):
        c = _result(out, (rows, n), dtype, device)
        rc = _g.lib().gemm_f16_grouped_nn(
            rows, groups, n, k, a.data_ptr(), b.data_ptr(), offsets.data_ptr(), c.data_ptr(), dtype is torch.float32, handle)
        if rc:
            raise _g.GemmError(rc)
        return c

    return _launch(device, stream, call)


def gemm_f16_grouped_tn(a, b, offsets, *, out_dtype=None, out=None, stream=None):
    """out[g] = a[rows of g].T @ b[rows of g]: a float16 [rows,K], b float16
    [rows,N], out [groups,K,N], zeros for an empty segment.  With a the
    gradient of gemm_f16_grouped_nt's output and b its rows, the gradient of
    its weights."""
    import torch

    dtype = _out_type(out_dtype)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("expected a [rows,K] and b [rows,N]")
    device = _first("a", a, torch.float16)
    (rows, k), n, groups = a.shape, b.shape[1], offsets.numel() - 1
    _operand("b", b, torch.float16, (rows, n), device)
    _operand("offsets", offsets, torch.int32, (groups + 1,), device)
    size = _workspace_bytes("gemm_f16_grouped_tn_workspace", rows, groups, n, k)

    def call(handle):
        c = _result(out, (groups, k, n), dtype, device)
        if size:
            ws = torch.empty(size, dtype=torch.uint8, device=device)
            rc = _g.lib().gemm_f16_grouped_tn_ws(
                rows, groups, n, k, a.data_ptr(), b.data_ptr(), offsets.data_ptr(), c.data_ptr(),
                dtype is torch.float32, ws.data_ptr(), size, handle)
        else:
            rc = _g.lib().gemm_f16_grouped_tn(
                rows, groups, n, k, a.data_ptr(), b.data_ptr(), offsets.data_ptr(), c.data_ptr(),
                dtype is torch.float32, handle)
        if rc:
            raise _g.GemmError(rc)
        return c

    return _launch(device, stream, call)


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
    device = _first("x", x, torch.float16)
    (rows, k), n, (adapters, rank, _) = x.shape, w.shape[0], down.shape
    _operand("w", w, torch.float16, (n, k), device)
    _operand("down", down, torch.float16, (adapters, rank, k), device)
    _operand("up", up, torch.float16, (adapters, n, rank), device)
    _operand("ids", ids, torch.int32, (rows,), device)
    _operand("order", order, torch.int32, (rows,), device)
    _operand("offsets", offsets, torch.int32, (adapters + 1,), device)
    if scale is not None:
        _operand("scale", scale, torch.float32, (adapters,), device)
    size = _workspace_bytes("gemm_f16_lora_workspace", rows, n, k, adapters, rank)

    def call(handle):
        y = _result(out, (rows, n), torch.float16, device)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        rc = _g.lib().gemm_f16_lora_nt(
            rows, n, k, adapters, rank, x.data_ptr(), w.data_ptr(), down.data_ptr(), up.data_ptr(), ids.data_ptr(),
            order.data_ptr(), offsets.data_ptr(), None if scale is None else scale.data_ptr(), y.data_ptr(),
            ws.data_ptr(), size, handle)
        if rc:
            raise _g.GemmError(rc)
        return y

    return _launch(device, stream, call)
