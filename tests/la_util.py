"""Plain fp64 forms of the decay linear attention, token by token, for its tests.

``forward`` and ``backward`` follow the definition (include/wkv7.h, wkv7_la_fwd and
wkv7_la_bwd) on any device.  ``bounds`` runs them on absolute values: the sums of the
magnitudes of all terms, which the rounding of a term or of a partial sum is relative to."""
import torch

U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24   # half a step of each type


def seqs(B, T, cu):
    """(batch row, first token, length) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, a, b - a) for a, b in zip(cu[:-1], cu[1:])]


def _bth(x, head_first):
    return x.transpose(1, 2) if head_first else x


def _inputs(q, k, v, g, mask, head_first, absolute):
    q, k, v = (_bth(x.double(), head_first) for x in (q, k, v))
    B, T, H = q.shape[:3]
    g = g.double()
    g = g.expand(B, T, H) if g.dim() == 1 else _bth(g, head_first)
    live = torch.ones(B, T, dtype=torch.bool, device=q.device) if mask is None else mask.bool()
    # what a masked token holds in k, v and g is not used
    k = torch.where(live[..., None, None], k, torch.zeros_like(k))
    v = torch.where(live[..., None, None], v, torch.zeros_like(v))
    g = torch.where(live[..., None], g, torch.zeros_like(g))
    if absolute:
        q, k, v = q.abs(), k.abs(), v.abs()
    return q, k, v, g, live


def forward(q, k, v, g, s0=None, mask=None, cu=None, scale=1.0, head_first=False,
            absolute=False):
    q, k, v, g, live = _inputs(q, k, v, g, mask, head_first, absolute)
    B, T, H, D = q.shape
    o = torch.zeros_like(q)
    finals = []
    for n, (b, a, L) in enumerate(seqs(B, T, cu)):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device)
        if s0 is not None:
            S = s0[n].double().abs() if absolute else s0[n].double()
        for t in range(a, a + L):
            S = torch.exp(g[b, t])[:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = (abs(scale) if absolute else scale) * torch.einsum("hkv,hk->hv", S, q[b, t])
        finals.append(S)
    return _bth(o, head_first), torch.stack(finals)


def backward(q, k, v, g, do, s0=None, mask=None, dsT=None, cu=None, scale=1.0, head_first=False,
             absolute=False, chunk_sums=False):
    """dq, dk, dv, dg ([H] when g is), ds0.  chunk_sums: dg as the sum of the magnitudes that
    a chunked evaluation adds (128-token chunks), for the bounds."""
    per_head = g.dim() == 1
    q, k, v, g, live = _inputs(q, k, v, g, mask, head_first, absolute)
    do = _bth(do.double(), head_first)
    if absolute:
        do, scale = do.abs(), abs(scale)
    B, T, H, D = q.shape
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    dg = torch.zeros(B, T, H, dtype=torch.float64, device=q.device)
    ds0 = []
    for n, (b, a, L) in enumerate(seqs(B, T, cu)):
        S = torch.zeros(H, D, D, dtype=torch.float64, device=q.device)
        if s0 is not None:
            S = s0[n].double().abs() if absolute else s0[n].double()
        states = [S]
        for t in range(a, a + L):
            S = torch.exp(g[b, t])[:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            states.append(S)
        G = torch.zeros_like(S)
        if dsT is not None:
            G = dsT[n].double().abs() if absolute else dsT[n].double()
        run = torch.zeros(H, dtype=torch.float64, device=q.device)
        for i in range(L - 1, -1, -1):
            t = a + i
            if chunk_sums and (i == L - 1 or i % 128 == 127):
                run = (states[i + 1] * G).sum((-1, -2))
            G = G + scale * q[b, t][:, :, None] * do[b, t][:, None, :]
            dq[b, t] = scale * torch.einsum("hkv,hv->hk", states[i + 1], do[b, t])
            if live[b, t]:
                dk[b, t] = torch.einsum("hkv,hv->hk", G, v[b, t])
                dv[b, t] = torch.einsum("hkv,hk->hv", G, k[b, t])
                dg[b, t] = torch.exp(g[b, t]) * (G * states[i]).sum((-1, -2))
            if chunk_sums:
                run = run + (q[b, t] * dq[b, t]).sum(-1) + (k[b, t] * dk[b, t]).sum(-1)
                if live[b, t]:
                    dg[b, t] = run
            G = torch.exp(g[b, t])[:, None, None] * G
        ds0.append(G)
    dg = dg.sum((0, 1)) if per_head else _bth(dg, head_first)
    return {"dq": _bth(dq, head_first), "dk": _bth(dk, head_first), "dv": _bth(dv, head_first),
            "dg": dg, "ds0": torch.stack(ds0)}


def allowed(ref, magnitude, dtype, length, D, tensor_cores, state=False):
    """Largest error that rounding can leave, element by element.

    fp32 sums and decays: a term passes at most `length` multiplications by decays (each
    with its own rounding and expf's, within 2 steps: 4 half steps) and length + D + 8 additions.  Tensor cores
    (bf16): scores, or the state before the chunk, enter a product once rounded to bf16, a
    half step of each term's magnitude, and the state's update operand in two bf16 parts
    (half a step of half a step).  Then the output's own rounding."""
    rel = (5 * length + D + 8) * U_F32
    if tensor_cores:
        rel += U_BF16 ** 2
        if not state:
            rel += U_BF16 * (1 + U_BF16)
    out = 0.0 if (state or dtype == torch.float32) else U_BF16
    return out * ref.abs() + rel * (1 + out) * magnitude


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst error "
        f"{float(torch.where(bad, err, torch.zeros_like(err)).max()):.3e}")
    n = float(ref.norm())
    return float((got.double() - ref).norm()) / n if n else 0.0
