"""Layer norm of rows, and of each head of a mixing layer's output, with its gradients.

``wkv7_ln_fwd`` and ``wkv7_ln_bwd`` marshal tensors to the entry points of the same names
(include/wkv7.h); ``layer_norm`` is the differentiable op.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .wkv7 import OK, WKV7Error, _check, _dtype_code, _ptr, _stream, library


def _groups(x, params, head_first):
    """Checks x and its weight and bias; returns rows, groups, inner, D and their type."""
    _check(x, "x")
    _dtype_code(x)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"x must have rows of 1 or more elements, got {tuple(x.shape)}")
    D = x.shape[-1]
    given = {n: t for n, t in params.items() if t is not None}
    shapes = {tuple(t.shape) for t in given.values()}
    dtypes = {t.dtype for t in given.values()}
    if len(shapes) > 1 or len(dtypes) > 1:
        raise ValueError(f"{', '.join(given)} must have one shape and one dtype")
    groups, inner = 1, 1
    wdtype = dtypes.pop() if dtypes else x.dtype
    if shapes:
        shape = shapes.pop()
        if len(shape) == 2:  # one weight and bias for each head
            groups = shape[0]
            if head_first:
                ok = x.dim() == 4 and x.shape[1] == groups
                inner = x.shape[2] if ok else 1
            else:
                ok = x.dim() >= 2 and x.shape[-2] == groups
            if not ok or groups == 0:
                raise ValueError(f"weight and bias {shape} do not fit x {tuple(x.shape)}")
        for n, t in given.items():
            _check(t, n, wdtype, (D,) if len(shape) != 2 else (groups, D))
            if t.device != x.device:
                raise ValueError(f"{n} is on {t.device}, x on {x.device}: one device only")
        if wdtype not in (torch.float32, x.dtype):
            raise TypeError(f"weights must be float32 or {x.dtype}, got {wdtype}")
    return x.numel() // D, groups, max(inner, 1), D, wdtype


def _code(dtype):
    return 0 if dtype == torch.bfloat16 else 1


def wkv7_ln_fwd(x, weight=None, bias=None, eps: float = 1e-5, head_first: bool = False, y=None):
    """Layer norm over the last dimension.  x [..., D] bf16 or fp32; weight, bias [D], or [H, D] for
    one of each head of x [..., H, D] (with head_first: of x [B, H, T, D]), in x's dtype or
    fp32, or None.  Returns (y, mean, rstd); the fp32 statistics have x's leading shape."""
    rows, groups, inner, D, wdtype = _groups(x, {"weight": weight, "bias": bias}, head_first)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(y, "y", x.dtype, x.shape)
        if y.device != x.device:
            raise ValueError(f"y is on {y.device}, x on {x.device}: one device only")
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    with torch.cuda.device(x.device):
        st = library().wkv7_ln_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean),
                                   _ptr(rstd), rows, groups, inner, D, float(eps),
                                   _dtype_code(x), _code(wdtype), _stream(x.device))
    if st != OK:
        raise WKV7Error(st, "wkv7_ln_fwd")
    return y, mean, rstd


def wkv7_ln_bwd(x, dy, mean, rstd, weight=None, head_first: bool = False, need_params=None,
                workspace=None):
    """Backward of wkv7_ln_fwd for L = sum(y * dy), with the forward's mean and rstd.  Returns a
    dict: dx, dweight, dbias (shaped like weight and in its dtype; None when there is no
    weight).  need_params False leaves dweight and dbias out."""
    rows, groups, inner, D, wdtype = _groups(x, {"weight": weight}, head_first)
    _check(dy, "dy", x.dtype, x.shape)
    _check(mean, "mean", torch.float32, x.shape[:-1])
    _check(rstd, "rstd", torch.float32, x.shape[:-1])
    for n, t in (("dy", dy), ("mean", mean), ("rstd", rstd), ("workspace", workspace)):
        if t is not None and t.device != x.device:
            raise ValueError(f"{n} is on {t.device}, x on {x.device}: one device only")
    need = (weight is not None) if need_params is None else bool(need_params)
    if need and weight is None:
        raise ValueError("need_params needs the weight")
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight) if need else None
    db = torch.empty_like(weight) if need else None
    lib = library()
    with torch.cuda.device(x.device):
        nbytes = int(lib.wkv7_ln_bwd_workspace_bytes(rows, groups, inner, D, _dtype_code(x)))
        if workspace is not None:
            _check(workspace, "workspace", torch.uint8)
        elif need and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        st = lib.wkv7_ln_bwd(_ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd), _ptr(weight), _ptr(dx),
                             _ptr(dw), _ptr(db), rows, groups, inner, D, _dtype_code(x),
                             _code(wdtype), _ptr(workspace),
                             0 if workspace is None else workspace.numel(), _stream(x.device))
    if st != OK:
        raise WKV7Error(st, "wkv7_ln_bwd")
    return {"dx": dx, "dweight": dw, "dbias": db}


class LayerNorm(torch.autograd.Function):
    """layer_norm as a differentiable op: wkv7_ln_fwd and wkv7_ln_bwd."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, head_first):
        y, mean, rstd = wkv7_ln_fwd(x, weight, bias, eps=eps, head_first=head_first)
        # the weight's gradient needs a weight to be shaped like; with a bias alone, ones
        ctx.ones = weight is None and bias is not None
        ctx.save_for_backward(x, torch.ones_like(bias) if ctx.ones else weight, mean, rstd)
        ctx.head_first = head_first
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        r = wkv7_ln_bwd(x, dy.to(x.dtype).contiguous(), mean, rstd, weight,
                        head_first=ctx.head_first,
                        need_params=ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
        dw = r["dweight"] if ctx.needs_input_grad[1] else None
        db = r["dbias"] if ctx.needs_input_grad[2] else None
        return r["dx"], dw, db, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, head_first: bool = False):
    """Differentiable layer norm; arguments as for wkv7_ln_fwd."""
    return LayerNorm.apply(x, weight, bias, eps, head_first)
