"""Layer norm forward and backward against their formulas in fp64, on the GPU; refusals on the
CPU; and the per-head norm inside the differentiable mixing ops.

Tolerances count roundings: a sum of D fp32 terms by a team of threads is a chain of at most
32 + 10 + 5 additions, so within 64 half steps (2^-24) of the sum of magnitudes; a bf16 result
adds its own half step (2^-8)."""
import ctypes

import pytest
import torch

import linear_attention_rnn_wkv7_b200 as lib
from linear_attention_rnn_wkv7_b200 import build as lib_build
from linear_attention_rnn_wkv7_b200.wkv7 import ERR_INVALID_ARG, ERR_UNSUPPORTED, OK

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
UB = 2.0 ** -8


def formula(x, w, b, eps):
    x = x.double()
    m = x.mean(-1, keepdim=True)
    r = ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - m) * r
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, m[..., 0], r[..., 0]


def gradients(x, dy, m, r, w, head_first=False):
    """dx, dw, db for given statistics; w [D], [H, D] or None."""
    x, dy, m, r = x.double(), dy.double(), m.double()[..., None], r.double()[..., None]
    xh = (x - m) * r
    wb = None if w is None else (w.double()[:, None] if head_first else w.double())
    u = dy if w is None else dy * wb
    dx = r * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    if w is None:
        return dx, None, None
    keep = w.dim() if not head_first else 2
    dims = (0, 2) if head_first else tuple(range(x.dim() - keep))
    return dx, (dy * xh).sum(dims), dy.sum(dims)


def make(shape, dtype, wshape, wdtype, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(*shape, generator=gen) + 1.5).to(dtype).cuda()
    dy = torch.randn(*shape, generator=gen).to(dtype).cuda()
    w = b = None
    if wshape:
        w = (1 + 0.3 * torch.randn(*wshape, generator=gen)).to(wdtype).cuda()
        b = torch.randn(*wshape, generator=gen).to(wdtype).cuda()
    return x, dy, w, b


def compare(x, dy, w, b, head_first=False, eps=1e-5):
    dtype = x.dtype
    out = UB if dtype == BF16 else U
    wr = w if w is None or not head_first else w[:, None]
    br = b if b is None or not head_first else b[:, None]
    y, mean, rstd = lib.wkv7_ln_fwd(x, w, b, eps=eps, head_first=head_first)
    ry, rm, rr = formula(x, wr, br, eps)
    mag = x.double().abs().mean(-1)
    em = 64 * U * mag
    assert bool(((mean.double() - rm).abs() <= em).all()), "mean"
    # the variance: 64 half steps of itself, and the mean's error against x - mean
    spread = (x.double() - rm[..., None]).abs().mean(-1)
    er = rr * (rr * rr * (64 * U / (rr * rr) + 2 * em * spread + em * em) + 8 * U)
    assert bool(((rstd.double() - rr).abs() <= er).all()), "rstd"
    xc = (x.double() - rm[..., None]).abs()
    wa = 1.0 if wr is None else wr.double().abs()
    ba = 0.0 if br is None else br.double().abs()
    tol = (wa * (xc * er[..., None] + rr[..., None] * (em[..., None] + U * x.double().abs()))
           + 4 * U * (wa * xc * rr[..., None] + ba))
    tol = tol * (1 + out) + out * ry.abs()
    assert bool(((y.double() - ry).abs() <= tol).all()), "y"

    g = lib.wkv7_ln_bwd(x, dy, mean, rstd, w, head_first=head_first)
    dx, dw, db = gradients(x, dy, mean, rstd, w, head_first)
    xh = (xc + U * x.double().abs()) * rr[..., None]
    u = dy.double().abs() * wa
    tol = rr[..., None] * 80 * U * (u + u.mean(-1, keepdim=True)
                                    + (xh + 1) * (u * (xh + 1)).mean(-1, keepdim=True))
    # xh itself is off by the rounding of x - mean
    ex = rr[..., None] * U * 3 * (x.double().abs() + mean.double().abs()[..., None])
    tol = tol + rr[..., None] * (ex * (u * xh).mean(-1, keepdim=True)
                                 + xh * (u * ex).mean(-1, keepdim=True))
    tol = tol * (1 + out) + out * dx.abs()
    assert bool(((g["dx"].double() - dx).abs() <= tol).all()), "dx"
    if w is None:
        assert g["dweight"] is None and g["dbias"] is None
        return
    wout = UB if w.dtype == BF16 else U
    keep = (0, 2) if head_first else tuple(range(x.dim() - w.dim()))
    rows = x.numel() // w.numel()
    sx, sd = (dy.double().abs() * (xh + ex)).sum(keep), dy.double().abs().sum(keep)
    n = (rows + 8) * U
    tol = n * sx + (dy.double().abs() * ex).sum(keep) + wout * dw.abs() * (1 + n)
    assert bool(((g["dweight"].double() - dw).abs() <= tol).all()), "dweight"
    tol = n * sd + wout * db.abs() * (1 + n)
    assert bool(((g["dbias"].double() - db).abs() <= tol).all()), "dbias"


# -------------------------------------------------------------------------- CPU: refusals
P = 0x7f0000000000


@pytest.fixture(scope="module")
def clib():
    lib_build.build()
    return lib.library()


def p(x):
    return ctypes.c_void_p(x)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), ERR_INVALID_ARG), (dict(x=P + 2), ERR_INVALID_ARG), (dict(y=P), ERR_INVALID_ARG),
    (dict(rows=-1), ERR_INVALID_ARG), (dict(D=0), ERR_INVALID_ARG),
    (dict(D=40000), ERR_UNSUPPORTED), (dict(groups=3), ERR_INVALID_ARG),
    (dict(groups=2, inner=3), ERR_INVALID_ARG), (dict(eps=-1.0), ERR_INVALID_ARG),
    (dict(eps=float("nan")), ERR_INVALID_ARG), (dict(dtype=1, wdtype=0), ERR_UNSUPPORTED),
    (dict(w=P + 4), ERR_INVALID_ARG), (dict(dtype=5), ERR_INVALID_ARG),
    (dict(inner=0), ERR_INVALID_ARG),
])
def test_fwd_refuses(clib, kw, status):
    a = dict(x=P, w=P + 4096, b=P + 8192, y=P + 65536, mean=0, rstd=0, rows=8, groups=1, inner=1,
             D=64, eps=1e-5, dtype=0, wdtype=0)
    a.update(kw)
    assert clib.wkv7_ln_fwd(p(a["x"]), p(a["w"]), p(a["b"]), p(a["y"]), p(a["mean"]),
                            p(a["rstd"]), a["rows"], a["groups"], a["inner"], a["D"], a["eps"],
                            a["dtype"], a["wdtype"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dy=0), ERR_INVALID_ARG), (dict(dx=P), ERR_INVALID_ARG), (dict(ws=0), ERR_INVALID_ARG),
    (dict(wsb=8), ERR_INVALID_ARG), (dict(mean=0), ERR_INVALID_ARG),
    (dict(dw=P + 2), ERR_INVALID_ARG), (dict(D=1 << 20), ERR_UNSUPPORTED),
    (dict(rows=7, groups=2), ERR_INVALID_ARG),
])
def test_bwd_refuses(clib, kw, status):
    a = dict(x=P, dy=P + 4096, mean=P + 8192, rstd=P + 16384, w=P + 32768, dx=P + 65536,
             dw=P + (1 << 20), db=P + (2 << 20), rows=8, groups=1, inner=1, D=64, dtype=0,
             wdtype=0, ws=P + (3 << 20), wsb=1 << 30)
    a.update(kw)
    assert clib.wkv7_ln_bwd(p(a["x"]), p(a["dy"]), p(a["mean"]), p(a["rstd"]), p(a["w"]),
                            p(a["dx"]), p(a["dw"]), p(a["db"]), a["rows"], a["groups"],
                            a["inner"], a["D"], a["dtype"], a["wdtype"], p(a["ws"]), a["wsb"],
                            None) == status


def test_binding_refuses():
    x = torch.randn(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        lib.wkv7_ln_fwd(x)
    with pytest.raises(ValueError, match="CUDA"):
        lib.layer_norm(x, torch.ones(64))


# ------------------------------------------------------------------------------ GPU: parity
SIZES = [1, 3, 8, 31, 64, 100, 129, 256, 500, 1000, 1021, 2048, 2050, 4096, 4100, 8191, 8192, 8200,
         10001, 16384, 20000, 32761, 32768]


@gpu
@pytest.mark.parametrize("D", SIZES)
@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_rows(cuda_device, D, dtype, wdtype):
    for rows in (1, 37):
        compare(*make((rows, D), dtype, (D,), wdtype, D + rows))
    compare(*make((5, D), dtype, None, wdtype, D))


@gpu
@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("D", [64, 100, 128, 256])
@pytest.mark.parametrize("H", [1, 3, 32])
@pytest.mark.parametrize("head_first", [False, True])
def test_heads(cuda_device, dtype, wdtype, D, H, head_first):
    shape = (2, H, 45, D) if head_first else (2, 45, H, D)
    compare(*make(shape, dtype, (H, D), wdtype, D + H), head_first=head_first)


@gpu
@pytest.mark.parametrize("D", [64, 1000, 4096])
def test_many_rows(cuda_device, D):
    """More rows than teams: a team's loop, and partial sums over many rows."""
    compare(*make((9001, D), BF16, (D,), F32, 3))


@gpu
def test_constant_and_huge_rows(cuda_device):
    """A constant row's y is 0 where its fp32 sums are exact (1000 and 2^60: up to 512 times either
    fits 24 bits).  1e18 rounds to a number of 24 significant bits, so three of it no longer
    fit: its mean may be off by the sum's roundings and its y is only bounded,
    |x - mean| <= sqrt(D) sqrt(mean of (x - mean)^2)."""
    x = torch.full((4, 512), 1000.0, device="cuda")
    x[1] = 1e18                                  # squares stay finite around the mean
    x[2, ::2] = -1000.0
    x[3] = 2.0 ** 60
    y, m, r = lib.wkv7_ln_fwd(x, eps=1e-5)
    want = torch.tensor([1000.0, 2.0 ** 60], device="cuda")
    assert torch.equal(m[[0, 3]], want) and bool((y[[0, 3]] == 0).all())
    assert abs(float(m[1]) / float(x[1, 0]) - 1) <= 64 * U
    assert bool((y[1].abs() <= 512 ** 0.5).all())
    assert bool(((y[2].abs() - 1).abs() < 1e-6).all())


@gpu
def test_empty(cuda_device):
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, m, r = lib.wkv7_ln_fwd(x, w, w)
    g = lib.wkv7_ln_bwd(x, x, m, r, w)
    assert y.shape == (0, 64) and torch.equal(g["dweight"], torch.zeros_like(w))


@gpu
def test_autograd_repeats_and_graphs(cuda_device):
    x, dy, w, b = make((300, 1000), BF16, (1000,), F32, 5)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = lib.layer_norm(*leaves)
    y.backward(dy)
    _, m, r = lib.wkv7_ln_fwd(x, w, b)
    g = lib.wkv7_ln_bwd(x, dy, m, r, w)
    for t, n in zip(leaves, ("dx", "dweight", "dbias")):
        assert torch.equal(t.grad, g[n]), n
    # a bias alone
    bias = b.clone().requires_grad_()
    lib.layer_norm(x, None, bias).backward(dy)
    assert torch.equal(bias.grad, g["dbias"])
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        y2, m2, r2 = lib.wkv7_ln_fwd(x, w, b)
        g2 = lib.wkv7_ln_bwd(x, dy, m2, r2, w)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, y.detach())
    for n in g:
        assert torch.equal(g[n], g2[n]), n


# ----------------------------------------------------------- GPU: inside the mixing layers
@gpu
@pytest.mark.parametrize("op", ["la", "gdn", "wkv7"])
@pytest.mark.parametrize("head_first", [False, True])
def test_norm_of_a_mixing_op(cuda_device, op, head_first):
    gen = torch.Generator().manual_seed(9)
    B, T, H, D = 2, 70, 3, 64
    lead = (B, H, T) if head_first else (B, T, H)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    q, k, v = r(*lead, D), torch.nn.functional.normalize(r(*lead, D), dim=-1), r(*lead, D)
    g = -torch.rand(*lead, generator=gen).cuda() * 0.5
    w, b = 1 + 0.1 * r(H, D), 0.1 * r(H, D)
    if op == "la":
        fn = lambda **kw: lib.decay_linear_attention(q, k, v, g, head_first=head_first, **kw)  # noqa: E731
    elif op == "gdn":
        fn = lambda **kw: lib.gated_delta_net(q, k, v, g, torch.sigmoid(g), head_first=head_first, **kw)  # noqa: E731,E501
    else:
        d = g[..., None].expand(*lead, D).contiguous()
        fn = lambda **kw: lib.generalized_delta_rule(q, d, k, v, -k, 0.5 * k, head_first=head_first, **kw)  # noqa: E731,E501
    o, s = fn()
    on, sn = fn(norm=(w, b, 1e-5))
    want, _, _ = lib.wkv7_ln_fwd(o, w, b, eps=1e-5, head_first=head_first)
    assert torch.equal(on, want) and torch.equal(s, sn)
    with pytest.raises(ValueError, match="norm"):
        fn(norm=(w[0].contiguous(), None, 1e-5))


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_of_all_operators(cuda_device, dtype):
    """Layer norm, the mixing with its per-head norm, backward through all of it, and tokens one
    by one after the prompt, against autograd of the formulas in fp64."""
    gen = torch.Generator().manual_seed(21)
    B, T, H, D = 2, 40, 2, 64
    C = H * D
    leaf = {"x": torch.randn(B, T, C, generator=gen), "w1": 1 + 0.1 * torch.randn(C, generator=gen),
            "b1": 0.1 * torch.randn(C, generator=gen), "w2": 1 + 0.1 * torch.randn(H, D, generator=gen),
            "b2": 0.1 * torch.randn(H, D, generator=gen),
            "g": -torch.rand(H, generator=gen) * 0.3}
    leaf = {n: t.to(dtype).cuda() for n, t in leaf.items()}
    mats = [(torch.randn(C, C, generator=gen) * C ** -0.5).to(dtype).cuda() for _ in range(3)]
    dy = torch.randn(B, T, H, D, generator=gen).to(dtype).cuda()

    a = {n: t.clone().requires_grad_() for n, t in leaf.items()}
    h = lib.layer_norm(a["x"], a["w1"], a["b1"])
    q, k, v = ((h @ m).view(B, T, H, D) for m in mats)
    o, state = lib.decay_linear_attention(q, k, v, a["g"], scale=D ** -0.5,
                                          norm=(a["w2"], a["b2"], 1e-3))
    o.backward(dy)

    c = {n: t.double().requires_grad_() for n, t in leaf.items()}
    hc = formula_grad(c["x"], c["w1"], c["b1"], 1e-5)
    qc, kc, vc = ((hc @ m.double()).view(B, T, H, D) for m in mats)
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda")
    outs = []
    for t in range(T):
        S = torch.exp(c["g"])[:, None, None] * S + kc[:, t][..., :, None] * vc[:, t][..., None, :]
        outs.append(D ** -0.5 * torch.einsum("bhkv,bhk->bhv", S, qc[:, t]))
    oc = formula_grad(torch.stack(outs, 1), c["w2"], c["b2"], 1e-3)
    oc.backward(dy.double())
    # a chain of about ten rounded stages, errors relative to each tensor's norm
    lim = 10 * (UB if dtype == BF16 else 64 * U)
    rel = lambda x, y: float(((x.double() - y).norm() / y.norm()).detach())  # noqa: E731
    assert rel(o, oc) <= lim
    assert rel(state, S) <= lim
    for n in leaf:
        assert rel(a[n].grad, c[n].grad) <= 2 * lim, n
    # the next token on the prompt's state
    y = lib.wkv7_la_step(*(t[:, -1].detach().contiguous() for t in (q, k, v)), a["g"].detach(),
                         state.detach().clone(), scale=D ** -0.5)
    z, _, _ = lib.wkv7_ln_fwd(y, leaf["w2"], leaf["b2"], eps=1e-3)
    S2 = torch.exp(c["g"])[:, None, None] * S + kc[:, -1][..., :, None] * vc[:, -1][..., None, :]
    yc = D ** -0.5 * torch.einsum("bhkv,bhk->bhv", S2, qc[:, -1])
    assert rel(z, formula_grad(yc, c["w2"], c["b2"], 1e-3)) <= lim
    assert lib.wkv7_get_last_error() == OK


def formula_grad(x, w, b, eps):
    m = x.mean(-1, keepdim=True)
    return (x - m) * ((x - m).square().mean(-1, keepdim=True) + eps).rsqrt() * w + b
