"""Linear attention with one decay per head: whole sequences, single tokens, gradients.

    S_t = e^{g_t} S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

``wkv7_la_fwd``, ``wkv7_la_step`` and ``wkv7_la_bwd`` marshal tensors to the entry points of
the same names (include/wkv7.h); ``decay_linear_attention`` is the differentiable op.
Tensors are dense and on one CUDA device; calls run on that device's current stream.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._args import address, expect, on_device, stream
from .wkv7 import ALGO, OK, WKV7Error, _check, _dense, _dtype_code, _head_norm, library


def _sizes(q, k, v, g, s0, mask, cu_seqlens, head_first):
    """Checks the inputs of a sequence call; returns B, T, H, K, V, N, g_per_head, mask."""
    _check(q, "q")
    _dtype_code(q)
    if q.dim() != 4:
        raise ValueError(f"q must have 4 dimensions, got {tuple(q.shape)}")
    if head_first:
        B, H, T, K = q.shape
    else:
        B, T, H, K = q.shape
    _check(v, "v", q.dtype)
    if v.dim() != 4:
        raise ValueError(f"v must have 4 dimensions, got {tuple(v.shape)}")
    V = v.shape[-1]
    expect(k, "k", q.dtype, q.shape, q)
    expect(v, "v", q.dtype, (*q.shape[:3], V), q)
    _check(g, "g", q.dtype)
    per_head = g.dim() == 1
    expect(g, "g", q.dtype, (H,) if per_head else q.shape[:3], q)
    N = B
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [N + 1]")
        expect(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, q)
        N = cu_seqlens.numel() - 1
    if s0 is not None:
        expect(s0, "s0", torch.float32, (N, H, K, V), q)
    if mask is not None:
        if mask.dtype == torch.bool:
            mask = mask.to(torch.uint8)
        expect(mask, "mask", torch.uint8, (B, T), q)
    return B, T, H, K, V, N, per_head, mask


def _workspace(given, nbytes, ref):
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=ref.device) if nbytes else None
    _check(given, "workspace", torch.uint8)
    expect(given, "workspace", torch.uint8, given.shape, ref)
    return given


def _zero_tail(x, scalars, T, H, K, cu_seqlens, N, head_first):
    """Zeros in the rows behind the last sequence of up to three fresh tensors and one of scalars."""
    x = list(x) + [None] * (3 - len(x))
    st = library().wkv7_la_zero_tail(*(address(t) for t in x), address(scalars), T, H, K,
                                     address(cu_seqlens), N, int(bool(head_first)),
                                     _dtype_code(x[0]), stream(x[0]))
    if st != OK:
        raise WKV7Error(st, "wkv7_la_zero_tail")


def wkv7_la_workspace_bytes(B, T, H, K=64, V=64, N=None, packed=False, dtype=torch.bfloat16,
                            algo: str = "auto", backward: bool = False) -> int:
    """Workspace bytes of wkv7_la_fwd or, with backward, of wkv7_la_bwd."""
    fn = (library().wkv7_la_bwd_workspace_bytes if backward
          else library().wkv7_la_fwd_workspace_bytes)
    return int(fn(B, T, H, K, V, B if N is None else N, int(packed),
                  0 if dtype == torch.bfloat16 else 1, ALGO[algo]))


def wkv7_la_fwd(q, k, v, g, s0=None, mask=None, cu_seqlens=None, output_final_state: bool = True,
                scale: float = 1.0, algo: str = "auto", o=None, sT=None,
                head_first: bool = False, workspace=None):
    """Linear attention with a decay for each head.  q, k [B,T,H,K]; v [B,T,H,V]; g [B,T,H] (log
    decay of each token) or [H] (of each head), bf16 or fp32, all alike; [B,H,T,*] and
    [B,H,T] with head_first; s0 [N,H,K,V] fp32 or None; mask [B,T] uint8/bool or None (0: the
    state stays); cu_seqlens [N+1] int32 from 0 (B must be 1) or None.  K = V in {64, 128, 256}.
    The workspace (uint8, wkv7_la_workspace_bytes) is allocated here when not given.  Rows behind
    the last packed sequence are 0 in an o that is allocated here and left alone in one given.
    Returns (o shaped like v, sT [N,H,K,V] fp32 or None)."""
    B, T, H, K, V, N, per_head, mask = _sizes(q, k, v, g, s0, mask, cu_seqlens, head_first)
    fresh = o is None
    if fresh:
        o = torch.empty_like(v)
    else:
        expect(o, "o", q.dtype, v.shape, q)
    if output_final_state and sT is None:
        sT = torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
    elif sT is not None:
        expect(sT, "sT", torch.float32, (N, H, K, V), q)
    lib = library()
    with on_device(q):
        need = int(lib.wkv7_la_fwd_workspace_bytes(B, T, H, K, V, N, int(cu_seqlens is not None),
                                                   _dtype_code(q), ALGO[algo]))
        ws = _workspace(workspace, need, q)
        st = lib.wkv7_la_fwd(address(q), address(k), address(v), address(g), int(per_head), address(s0),
                             address(mask), address(o), address(sT), B, T, H, K, V, address(cu_seqlens), N,
                             float(scale), int(bool(head_first)), _dtype_code(q), ALGO[algo],
                             address(ws), 0 if ws is None else ws.numel(), stream(q))
        if st == OK and fresh and cu_seqlens is not None:
            _zero_tail([o], None, T, H, K, cu_seqlens, N, head_first)
    if st != OK:
        raise WKV7Error(st, "wkv7_la_fwd")
    return o, sT


def wkv7_la_step(q, k, v, g, state, out_state=None, scale: float = 1.0, o=None):
    """One decode token.  q, k [B,H,K]; v [B,H,V]; g [B,H] or [H]; state [B,H,K,V] fp32, updated
    in place unless out_state takes the new one.  Returns o [B,H,V]."""
    _check(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dimensions, got {tuple(q.shape)}")
    B, H, K = q.shape
    V = v.shape[-1]
    expect(k, "k", q.dtype, (B, H, K), q)
    expect(v, "v", q.dtype, (B, H, V), q)
    per_head = g.dim() == 1
    expect(g, "g", q.dtype, (H,) if per_head else (B, H), q)
    expect(state, "state", torch.float32, (B, H, K, V), q)
    if out_state is None:
        out_state = state
    else:
        expect(out_state, "out_state", torch.float32, (B, H, K, V), q)
    if o is None:
        o = torch.empty_like(v)
    else:
        expect(o, "o", q.dtype, (B, H, V), q)
    with on_device(q):
        st = library().wkv7_la_step(address(q), address(k), address(v), address(g), int(per_head),
                                    address(state), address(out_state), address(o), B, H, K, V,
                                    float(scale), _dtype_code(q), stream(q))
    if st != OK:
        raise WKV7Error(st, "wkv7_la_step")
    return o


def wkv7_la_bwd(q, k, v, g, dout, s0=None, mask=None, dsT=None, cu_seqlens=None,
                scale: float = 1.0, algo: str = "auto", head_first: bool = False, workspace=None,
                need_dg: bool = True, need_ds0: bool = True):
    """Backward of wkv7_la_fwd for L = sum(o * dout) + sum(S_T * dsT).  Returns a dict: dq, dk, dv,
    dg (input dtype, shaped like the inputs; dg of a [H] g is summed over batch and tokens) and
    ds0 (fp32 [N,H,K,V]); dg and ds0 are None when not needed.  Rows behind the last packed
    sequence have gradients of 0."""
    B, T, H, K, V, N, per_head, mask = _sizes(q, k, v, g, s0, mask, cu_seqlens, head_first)
    expect(dout, "dout", q.dtype, v.shape, q)
    if dsT is not None:
        expect(dsT, "dsT", torch.float32, (N, H, K, V), q)
    lib = library()
    with on_device(q):
        need = int(lib.wkv7_la_bwd_workspace_bytes(B, T, H, K, V, N, int(cu_seqlens is not None),
                                                   _dtype_code(q), ALGO[algo]))
        ws = _workspace(workspace, need, q)
        out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
               "dg": torch.empty_like(g) if need_dg else None,
               "ds0": torch.empty((N, H, K, V), dtype=torch.float32, device=q.device)
               if need_ds0 else None}
        st = lib.wkv7_la_bwd(address(q), address(k), address(v), address(g), int(per_head), address(s0),
                             address(mask), address(dout), address(dsT), address(out["dq"]), address(out["dk"]),
                             address(out["dv"]), address(out["dg"]), address(out["ds0"]), B, T, H, K, V,
                             address(cu_seqlens), N, float(scale), int(bool(head_first)),
                             _dtype_code(q), ALGO[algo], address(ws),
                             0 if ws is None else ws.numel(), stream(q))
        if st == OK and cu_seqlens is not None:
            _zero_tail([out["dq"], out["dk"], out["dv"]], None if per_head else out["dg"], T, H, K,
                       cu_seqlens, N, head_first)
    if st != OK:
        raise WKV7Error(st, "wkv7_la_bwd")
    return out


class DecayLinearAttention(torch.autograd.Function):
    """decay_linear_attention as a differentiable op: wkv7_la_fwd and wkv7_la_bwd."""

    @staticmethod
    def forward(ctx, q, k, v, g, s0, mask, cu_seqlens, scale, head_first, final, algo):
        o, sT = wkv7_la_fwd(q, k, v, g, s0=s0, mask=mask, cu_seqlens=cu_seqlens,
                            output_final_state=final, scale=scale, algo=algo,
                            head_first=head_first)
        ctx.save_for_backward(q, k, v, g, s0, mask, cu_seqlens)
        ctx.scale, ctx.head_first, ctx.algo = scale, head_first, algo
        ctx.set_materialize_grads(False)
        return o, sT

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dsT):
        q, k, v, g, s0, mask, cu_seqlens = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else _dense(do, v.dtype)
        dsT = None if dsT is None else _dense(dsT, torch.float32)
        r = wkv7_la_bwd(q, k, v, g, do, s0=s0, mask=mask, dsT=dsT, cu_seqlens=cu_seqlens,
                        scale=ctx.scale, algo=ctx.algo, head_first=ctx.head_first,
                        need_dg=ctx.needs_input_grad[3], need_ds0=ctx.needs_input_grad[4])
        return (r["dq"], r["dk"], r["dv"], r["dg"], r["ds0"], *[None] * 6)


def decay_linear_attention(q, k, v, g, initial_state=None, output_final_state: bool = True,
                           mask=None, cu_seqlens=None, scale: float = 1.0,
                           head_first: bool = False, norm=None, algo: str = "auto"):
    """Differentiable linear attention with a decay for each head; arguments as for
    wkv7_la_fwd, norm = (weight, bias, eps) as for generalized_delta_rule.  For bf16 the tensor
    cores' scores and state copies are bf16 too (o is 2.34e-3 off, rounding it alone 1.66e-3);
    algo = "recurrent" keeps everything but the results in fp32 and takes longer (8 x 4096 tokens
    of 64 heads of 64: forward 4.7 ms for 0.29 ms, backward 13.9 ms for 1.26 ms).  Returns (o,
    final state or None)."""
    o, sT = DecayLinearAttention.apply(q, k, v, g, initial_state, mask, cu_seqlens, scale,
                                       head_first, output_final_state, algo)
    return _head_norm(o, norm, head_first), sT
