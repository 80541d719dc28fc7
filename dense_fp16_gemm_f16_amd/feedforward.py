"""The feed-forward layer around the products, dense and routed.

* ``gemm_f16_fused_nt``    act(A B^T + bias) + residual
* ``gemm_f16_fused_grad``  dz = dy act'(z) and the bias's gradient
* ``route``                logits -> each token's experts and gates
* ``route_grad``           the logits' gradient from the gates'
* ``combine_rows``         the experts' rows, weighted, back to their tokens
* ``combine_rows_grad``    its gradients by the rows and the gates

Every call is asynchronous on ``stream`` (default: torch's current stream),
never waits for the GPU and captures into HIP graphs, as the segmented
products do (segments.py); the arguments' contracts are those of
``include/gemm_f16.h``.
"""
from __future__ import annotations

import ctypes

import dense_fp16_gemm_f16_amd as _g

from .segments import _first, _launch, _operand, _out_type, _result, _workspace_bytes

ACTS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
SCORES = {"softmax": 0, "sigmoid": 1}


class Epilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("bias_f32", ctypes.c_int32), ("out_f32", ctypes.c_int32),
                ("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("pre", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


def _act(name):
    if name not in ACTS:
        raise ValueError(f"act must be one of {', '.join(str(a) for a in ACTS)}")
    return ACTS[name]


def _float_type(name, t):
    import torch

    if t.dtype is not torch.float16 and t.dtype is not torch.float32:
        raise TypeError(f"{name} must be float16 or float32")
    return t.dtype


def _ptr(t):
    return None if t is None else t.data_ptr()


def _buffer(size, device):
    import torch

    return torch.empty(size, dtype=torch.uint8, device=device) if size else None


def gemm_f16_fused_nt(a, b, bias=None, *, act=None, residual=None, return_pre: bool = False, out_dtype=None, out=None,
                      stream=None):
    """act(a @ b.T + bias) + residual in one kernel: a float16 [M,K], b float16 [N,K].

    ``act``: None, "relu", "gelu" (erf), "gelu_tanh" or "silu".  ``bias`` [N]
    float16 or float32; ``residual`` [M,N] of the output's type, which
    ``out_dtype`` sets (float16, the default, or float32); ``out`` may be
    ``residual`` itself.  With ``return_pre`` the result is (out, pre), pre =
    a @ b.T + bias in float16, which gemm_f16_fused_grad takes.
    """
    import torch

    dtype, code = _out_type(out_dtype), _act(act)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("expected a [M,K] and b [N,K]")
    device = _first("a", a, torch.float16)
    (m, k), n = a.shape, b.shape[0]
    _operand("b", b, torch.float16, (n, k), device)
    if bias is not None:
        _operand("bias", bias, _float_type("bias", bias), (n,), device)
    if residual is not None:
        _operand("residual", residual, dtype, (m, n), device)
    size = _workspace_bytes("gemm_f16_fused_workspace", m, n, k)

    def call(handle):
        c = _result(out, (m, n), dtype, device)
        pre = torch.empty(m, n, dtype=torch.float16, device=device) if return_pre else None
        ws = _buffer(size, device)
        e = Epilogue(code, bias is not None and bias.dtype is torch.float32, dtype is torch.float32, _ptr(bias),
                     _ptr(residual), _ptr(pre))
        rc = _g.lib().gemm_f16_fused_nt(m, n, k, a.data_ptr(), b.data_ptr(), c.data_ptr(), ctypes.byref(e), _ptr(ws), size, handle)
        if rc:
            raise _g.GemmError(rc)
        return (c, pre) if return_pre else c

    return _launch(device, stream, call)


def gemm_f16_fused_grad(dy, pre=None, *, act=None, bias_grad: bool = True, stream=None):
    """(dz, dbias) of gemm_f16_fused_nt from dy, the gradient of its output.

    dy [M,N] float16 or float32; ``pre`` float16 [M,N] of the forward call (not
    needed without ``act``).  dz = dy * act'(pre) is float16, the operand of
    the products that give the gradients of a (dz @ b) and b (dz.T @ a);
    without ``act`` it is dy itself.  dbias float32 [N] sums dz before its
    rounding, or is None (``bias_grad`` False).
    """
    import torch

    code = _act(act)
    dtype = _float_type("dy", dy)
    if dy.dim() != 2:
        raise ValueError("expected dy [M,N]")
    device = _first("dy", dy, dtype)
    m, n = dy.shape
    if act is not None:
        if pre is None:
            raise ValueError("pre is needed with an activation")
        _operand("pre", pre, torch.float16, (m, n), device)
    size = _workspace_bytes("gemm_f16_fused_grad_workspace", m, n) if bias_grad else 0

    def call(handle):
        dz = torch.empty(m, n, dtype=torch.float16, device=device) if act is not None else None
        dbias = torch.empty(n, dtype=torch.float32, device=device) if bias_grad else None
        ws = _buffer(size, device)
        rc = _g.lib().gemm_f16_fused_grad(m, n, dy.data_ptr(), dtype is torch.float32, None if act is None else pre.data_ptr(),
                                          code, _ptr(dz), _ptr(dbias), _ptr(ws), size, handle)
        if rc:
            raise _g.GemmError(rc)
        return dy if dz is None else dz, dbias

    return _launch(device, stream, call)


def _routing(score, groups, top_groups, group_top, renormalize, scale, fan=1):
    if score not in SCORES:
        raise ValueError(f"score must be one of {', '.join(SCORES)}")
    # (here too, as results of such a size are not allocated, and ctypes drops the bits past 32)
    if not (1 <= fan <= 32 and 1 <= groups <= 64 and 1 <= top_groups <= 64 and 1 <= group_top <= 2):
        raise _g.GemmError(_g.EINVAL)
    return Routing(SCORES[score], groups, top_groups, group_top, bool(renormalize), scale)


def route(logits, fan: int, *, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1, group_top: int = 1,
          renormalize: bool = True, scale: float = 1.0, stream=None):
    """Each token's experts and gates from its logits: (ids, gates), int32 and
    float32 [tokens, fan].

    logits [tokens, experts] float16 or float32.  Scores are ``score``
    ("softmax" or "sigmoid") of the logits; the ``fan`` experts of largest
    score + ``bias`` (float32 [experts], for the choice only) are taken in
    falling order, ties to the lowest index.  With ``groups`` > 1 neighbouring
    experts form groups, and only the ``top_groups`` with the largest value are
    open: their largest score + bias (``group_top`` 1) or the sum of their two
    largest (2).  gates are ``scale`` times the scores, divided by their sum
    with ``renormalize``.  Experts whose logit or score + bias is -inf or NaN
    are never taken; where too few are left, ids are -1 (which ``group_rows``
    sorts behind all experts) and gates 0.
    """
    import torch

    dtype = _float_type("logits", logits)
    if logits.dim() != 2:
        raise ValueError("expected logits [tokens, experts]")
    r = _routing(score, groups, top_groups, group_top, renormalize, scale, fan)
    device = _first("logits", logits, dtype)
    tokens, experts = logits.shape
    if bias is not None:
        _operand("bias", bias, torch.float32, (experts,), device)

    def call(handle):
        ids = torch.empty(tokens, fan, dtype=torch.int32, device=device)
        gates = torch.empty(tokens, fan, dtype=torch.float32, device=device)
        rc = _g.lib().gemm_f16_route(tokens, experts, fan, logits.data_ptr(), dtype is torch.float32, _ptr(bias), ctypes.byref(r),
                                     ids.data_ptr(), gates.data_ptr(), handle)
        if rc:
            raise _g.GemmError(rc)
        return ids, gates

    return _launch(device, stream, call)


def route_grad(logits, ids, dgates, *, score: str = "softmax", renormalize: bool = True, scale: float = 1.0, stream=None):
    """The gradient of route's logits, of their type, from that of its gates:
    ids int32 and dgates float32 [tokens, fan]; the choice is held fixed."""
    import torch

    dtype = _float_type("logits", logits)
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError("expected logits [tokens, experts] and ids [tokens, fan]")
    device = _first("logits", logits, dtype)
    (tokens, experts), fan = logits.shape, ids.shape[1]
    _operand("ids", ids, torch.int32, (tokens, fan), device)
    _operand("dgates", dgates, torch.float32, (tokens, fan), device)
    r = _routing(score, 1, 1, 1, renormalize, scale)

    def call(handle):
        dlogits = torch.empty(tokens, experts, dtype=dtype, device=device)
        rc = _g.lib().gemm_f16_route_grad(tokens, experts, fan, logits.data_ptr(), dtype is torch.float32, ids.data_ptr(),
                                          dgates.data_ptr(), ctypes.byref(r), dlogits.data_ptr(), handle)
        if rc:
            raise _g.GemmError(rc)
        return dlogits

    return _launch(device, stream, call)


def _plan(rows, inverse, offsets, fan, dtype):
    """Sizes of a routed batch and its operands' device."""
    import torch

    shape, ends = rows.shape, offsets.shape
    if len(shape) != 2 or len(ends) != 1 or ends[0] < 2:
        raise ValueError("expected rows [tokens * fan, N] and offsets [groups + 1]")
    places, n = shape
    if fan < 1 or places % fan != 0:
        raise ValueError("rows must hold fan rows of each token")
    device = _first("rows", rows, dtype)
    _operand("inverse", inverse, torch.int32, (places,), device)
    _operand("offsets", offsets, torch.int32, ends, device)
    return places // fan, n, ends[0] - 1, device


def combine_rows(rows, inverse, offsets, fan: int, *, gates=None, residual=None, out_dtype=None, out=None, stream=None):
    """out[t] = residual[t] + sum_f gates[t, f] * rows[inverse[t * fan + f]].

    rows [tokens * fan, N] float16 or float32, in the order of (_, inverse,
    offsets) = group_rows(ids, groups) of ids [tokens, fan]; ``gates`` float32
    [tokens, fan] (default: ones, which gives the gradient of gathered tokens
    from that of their rows).  Rows from offsets[-1] on add nothing.
    ``residual`` [tokens, N] is of the output's type (``out_dtype`` float16,
    the default, or float32) and may be ``out`` itself.
    """
    import torch

    dtype, rows_type = _out_type(out_dtype), _float_type("rows", rows)
    tokens, n, groups, device = _plan(rows, inverse, offsets, fan, rows_type)
    if gates is not None:
        _operand("gates", gates, torch.float32, (tokens, fan), device)
    if residual is not None:
        _operand("residual", residual, dtype, (tokens, n), device)

    def call(handle):
        y = _result(out, (tokens, n), dtype, device)
        rc = _g.lib().gemm_f16_combine_rows(tokens, fan, n, groups, rows.data_ptr(), rows_type is torch.float32,
                                            inverse.data_ptr(), offsets.data_ptr(), _ptr(gates), _ptr(residual), y.data_ptr(),
                                            dtype is torch.float32, handle)
        if rc:
            raise _g.GemmError(rc)
        return y

    return _launch(device, stream, call)


def combine_rows_grad(dy, rows, inverse, offsets, gates, *, rows_dtype=None, stream=None):
    """(drows, dgates) of combine_rows from dy, the gradient of its output:
    drows [tokens * fan, N] of ``rows_dtype`` (float16, the default: the operand
    of the experts' gradient products; or float32), dgates float32 [tokens,
    fan].  The residual's gradient is dy."""
    import torch

    dtype, dy_type, rows_type = _out_type(rows_dtype), _float_type("dy", dy), _float_type("rows", rows)
    if gates.dim() != 2:
        raise ValueError("expected gates [tokens, fan]")
    fan = gates.shape[1]
    tokens, n, groups, device = _plan(rows, inverse, offsets, fan, rows_type)
    _operand("dy", dy, dy_type, (tokens, n), device)
    _operand("gates", gates, torch.float32, (tokens, fan), device)

    def call(handle):
        drows = torch.empty(tokens * fan, n, dtype=dtype, device=device)
        dgates = torch.empty(tokens, fan, dtype=torch.float32, device=device)
        rc = _g.lib().gemm_f16_combine_rows_grad(tokens, fan, n, groups, dy.data_ptr(), dy_type is torch.float32, rows.data_ptr(),
                                                 rows_type is torch.float32, inverse.data_ptr(), offsets.data_ptr(),
                                                 gates.data_ptr(), drows.data_ptr(), dtype is torch.float32, dgates.data_ptr(),
                                                 handle)
        if rc:
            raise _g.GemmError(rc)
        return drows, dgates

    return _launch(device, stream, call)
