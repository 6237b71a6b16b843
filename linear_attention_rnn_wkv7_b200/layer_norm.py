"""Layer norm of rows, and of each head of a mixing layer's output, with its gradients.

``wkv7_ln_fwd`` and ``wkv7_ln_bwd`` marshal tensors to the entry points of the same names
(include/wkv7.h); ``layer_norm`` is the differentiable op.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._args import address, expect, on_device, stream
from .wkv7 import OK, WKV7Error, _check, _dense, _dtype_code, library


def _groups(x, params, head_first):
    """Checks x and its weight and bias; returns rows, groups, inner, D and their type."""
    _check(x, "x")
    _dtype_code(x)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError(f"x must have rows of 1 or more elements, got {tuple(x.shape)}")
    D = x.shape[-1]
    groups, inner, shape, wdtype = 1, 1, None, x.dtype
    for n, t in params:
        if t is None:
            continue
        if shape is None:
            shape, wdtype = t.shape, t.dtype
            if len(shape) == 2:  # one weight and bias for each head
                groups = shape[0]
                if head_first:
                    ok = x.dim() == 4 and x.shape[1] == groups
                    inner = x.shape[2] if ok else 1
                else:
                    ok = x.dim() >= 2 and x.shape[-2] == groups
                if not ok or groups == 0:
                    raise ValueError(f"{n} {tuple(shape)} does not fit x {tuple(x.shape)}")
            if wdtype is not x.dtype and wdtype is not torch.float32:
                raise TypeError(f"{n} must be float32 or {x.dtype}, got {wdtype}")
            expect(t, n, wdtype, (groups, D) if len(shape) == 2 else (D,), x)
        else:
            expect(t, n, wdtype, shape, x)
    return x.numel() // D, groups, max(inner, 1), D, wdtype


def _code(dtype):
    return 0 if dtype == torch.bfloat16 else 1


def wkv7_ln_fwd(x, weight=None, bias=None, eps: float = 1e-5, head_first: bool = False, y=None):
    """Layer norm over the last dimension.  x [..., D] bf16 or fp32; weight, bias [D], or [H, D] for
    one of each head of x [..., H, D] (with head_first: of x [B, H, T, D]), in x's dtype or
    fp32, or None.  Returns (y, mean, rstd); the fp32 statistics have x's leading shape."""
    rows, groups, inner, D, wdtype = _groups(x, (("weight", weight), ("bias", bias)), head_first)
    if y is None:
        y = torch.empty_like(x)
    else:
        expect(y, "y", x.dtype, x.shape, x)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    with on_device(x):
        st = library().wkv7_ln_fwd(address(x), address(weight), address(bias), address(y), address(mean),
                                   address(rstd), rows, groups, inner, D, float(eps),
                                   _dtype_code(x), _code(wdtype), stream(x))
    if st != OK:
        raise WKV7Error(st, "wkv7_ln_fwd")
    return y, mean, rstd


def wkv7_ln_bwd(x, dy, mean, rstd, weight=None, head_first: bool = False, need_params=None,
                workspace=None):
    """Backward of wkv7_ln_fwd for L = sum(y * dy), with the forward's mean and rstd.  Returns a
    dict: dx, dweight, dbias (shaped like weight and in its dtype; None when there is no
    weight).  need_params False leaves dweight and dbias out."""
    rows, groups, inner, D, wdtype = _groups(x, (("weight", weight),), head_first)
    expect(dy, "dy", x.dtype, x.shape, x)
    expect(mean, "mean", torch.float32, x.shape[:-1], x)
    expect(rstd, "rstd", torch.float32, x.shape[:-1], x)
    need = (weight is not None) if need_params is None else bool(need_params)
    if need and weight is None:
        raise ValueError("need_params needs the weight")
    dx = torch.empty_like(x)
    dw = torch.empty_like(weight) if need else None
    db = torch.empty_like(weight) if need else None
    lib = library()
    with on_device(x):
        nbytes = int(lib.wkv7_ln_bwd_workspace_bytes(rows, groups, inner, D, _dtype_code(x)))
        if workspace is not None:
            expect(workspace, "workspace", torch.uint8, workspace.shape, x)
        elif need and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        st = lib.wkv7_ln_bwd(address(x), address(dy), address(mean), address(rstd), address(weight), address(dx),
                             address(dw), address(db), rows, groups, inner, D, _dtype_code(x),
                             _code(wdtype), address(workspace),
                             0 if workspace is None else workspace.numel(), stream(x))
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
        r = wkv7_ln_bwd(x, _dense(dy, x.dtype), mean, rstd, weight,
                        head_first=ctx.head_first,
                        need_params=ctx.needs_input_grad[1] or ctx.needs_input_grad[2])
        dw = r["dweight"] if ctx.needs_input_grad[1] else None
        db = r["dbias"] if ctx.needs_input_grad[2] else None
        return r["dx"], dw, db, None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, head_first: bool = False):
    """Differentiable layer norm; arguments as for wkv7_ln_fwd."""
    return LayerNorm.apply(x, weight, bias, eps, head_first)
