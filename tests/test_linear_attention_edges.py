"""The decay linear attention where states are carried far, rows lie behind the last sequence or
gradients arrive as views: cases of their own beside test_linear_attention.py."""
import pytest
import torch

import la_util as ref
import linear_attention_rnn_wkv7_b200 as lib
from linear_attention_rnn_wkv7_b200.wkv7 import OK

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


# ------------------------------------------------------------- states carried by strong decays
SHAPES = [(2, 300, 64), (40, 300, 4), (1, 1500, 2), (3, 300, 2)]  # rounds, runs, segments, few


@pytest.mark.parametrize("algo", ["auto", "recurrent"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,T,H", SHAPES)
@pytest.mark.parametrize("strong", [-0.078125, -0.1015625, -0.1171875, -0.25, -0.5])
def test_state_carried_through_a_strong_chunk(cuda_device, algo, D, B, T, H, strong):
    """With nothing added (k = 0, q = 0) the final state is e^{sum of g} s0, and ds0 the same of
    dsT, each entry relative to itself.  One chunk of 128 tokens decays by e^{128 strong}.

    A sum of a chunk's decays (all of one sign) passes 10 roundings at most on its way, with the
    factor log2(e) and a segment's sum over its chunks chunks + 2 more, each half a step of at
    most |sum|; an exponential is within 4 half steps, and each chunk or segment multiplies once."""
    gen = torch.Generator().manual_seed(B + T)
    q, k = torch.zeros(B, T, H, D, dtype=BF16, device="cuda"), torch.zeros(B, T, H, D, dtype=BF16, device="cuda")
    v, do = (torch.randn(B, T, H, D, generator=gen).to(BF16).cuda() for _ in range(2))
    g = torch.full((B, T, H), -2.0 ** -9, dtype=BF16, device="cuda")
    g[:, 128:256] = strong
    s0, dsT = (torch.randn(B, H, D, D, generator=gen).cuda() for _ in range(2))
    _, sT = lib.wkv7_la_fwd(q, k, v, g, s0=s0, algo=algo)
    ds0 = lib.wkv7_la_bwd(q, k, v, g, do, s0=s0, dsT=dsT, algo=algo)["ds0"]
    total = g.double().sum(1)[..., None, None]
    chunks = (T + 127) // 128
    if algo == "recurrent":
        chunks = T   # a product for each token
    tol = ((12 + chunks) * total.abs() + 5 * (2 * chunks + 2)) * U
    for got, start, name in ((sT, s0, "sT"), (ds0, dsT, "ds0")):
        want = start.double() * total.exp()
        bad = (got.double() - want).abs() > tol * want.abs()
        assert not bool(bad.any()), (name, float(((got.double() - want) / want).abs().max()),
                                     float(tol.max()))
    assert lib.wkv7_get_last_error() == OK


# --------------------------------------------------------------- rows behind the last sequence
def dirty(*like):
    """Leaves NaN in memory that the next allocations of these shapes are likely to get."""
    for t in like:
        for _ in range(4):
            torch.full_like(t, float("nan"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("head_first", [False, True])
@pytest.mark.parametrize("cu", [[0, 70, 200], [0, 0, 0], [0], [0, 200, 333]])
def test_rows_behind_the_last_sequence_are_zero(cuda_device, dtype, D, head_first, cu):
    """What the binding allocates is defined everywhere: no output and no gradient behind the last
    sequence, so that the norm behind it and the layers before it stay finite."""
    gen = torch.Generator().manual_seed(4)
    T, H, end = 333, 3, cu[-1]
    lead = (1, H, T) if head_first else (1, T, H)
    x = {n: torch.randn(*lead, D, generator=gen).to(dtype).cuda() for n in ("q", "k", "v", "do")}
    x["g"] = -torch.rand(*lead, generator=gen).to(dtype).cuda()
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    rows = (lambda t: t.transpose(1, 2)) if head_first else (lambda t: t)
    dirty(*x.values())
    o, _ = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu_t, head_first=head_first)
    assert bool((rows(o)[:, end:] == 0).all())
    dirty(*x.values())
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu_t,
                        head_first=head_first)
    for n in ("dq", "dk", "dv", "dg"):
        assert bool((rows(r[n])[:, end:] == 0).all()), n

    w, b = (torch.randn(H, D, generator=gen).cuda() for _ in range(2))
    a = {n: t.clone().requires_grad_() for n, t in {**x, "w": w, "b": b}.items() if n != "do"}
    dirty(*x.values())
    y, _ = lib.decay_linear_attention(a["q"], a["k"], a["v"], a["g"], cu_seqlens=cu_t,
                                      head_first=head_first, norm=(a["w"], a["b"], 1e-5))
    dirty(*x.values())
    rows(y)[:, :end].backward(rows(x["do"])[:, :end])
    for n, t in a.items():
        assert bool(torch.isfinite(t.grad).all()), n
    for n in ("q", "k", "v", "g"):
        assert bool((rows(a[n].grad)[:, end:] == 0).all()), n
    assert lib.wkv7_get_last_error() == OK


# ------------------------------------------------------------------- gradients that are views
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("op", ["la", "gdn", "wkv7"])
def test_gradient_that_is_a_shifted_view(cuda_device, op, dtype):
    """Outputs joined behind an odd number of elements get gradients that are dense but not
    16-byte aligned; they give what aligned copies of them give."""
    gen = torch.Generator().manual_seed(6)
    B, T, H, D = 1, 70, 2, 64
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    q, v = r(B, T, H, D).requires_grad_(), r(B, T, H, D).requires_grad_()
    k = torch.nn.functional.normalize(r(B, T, H, D).float(), dim=-1).to(dtype)
    g = -torch.rand(B, T, H, generator=gen).to(dtype).cuda()
    if op == "la":
        o, s = lib.decay_linear_attention(q, k, v, g)
    elif op == "gdn":
        o, s = lib.gated_delta_net(q, k, v, g, torch.sigmoid(g))
    else:
        o, s = lib.generalized_delta_rule(q, g[..., None].expand(B, T, H, D).contiguous(), k, v, -k,
                                          0.5 * k)
    do, ds = r(o.numel() + 1), torch.randn(s.numel() + 1, generator=gen).cuda()
    want = torch.autograd.grad((o, s), (q, v), (do[1:].clone().view_as(o), ds[1:].clone().view_as(s)),
                               retain_graph=True)
    one, onef = torch.zeros(1, dtype=dtype, device="cuda"), torch.zeros(1, device="cuda")
    joined, states = torch.cat([one, o.flatten()]), torch.cat([onef, s.flatten()])
    got = torch.autograd.grad((joined, states), (q, v), (do, ds))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------- the differentiable op's algorithm
@pytest.mark.parametrize("D", [64, 128])
def test_op_takes_the_algorithm(cuda_device, D):
    """algo reaches both directions: "recurrent" holds all but the results in fp32, so each is off by
    its own rounding (at most 2^-8 of a value) and fp32's, also where the tensor cores are not."""
    gen = torch.Generator().manual_seed(D)
    B, T, H = 2, 200, 3
    x = {n: torch.randn(B, T, H, D, generator=gen).to(BF16).cuda() for n in ("q", "k", "v", "do")}
    x["g"] = -torch.rand(B, T, H, generator=gen).to(BF16).cuda() * 0.1
    want, _ = ref.forward(x["q"], x["k"], x["v"], x["g"], scale=D ** -0.5)
    size, _ = ref.forward(x["q"], x["k"], x["v"], x["g"], scale=D ** -0.5, absolute=True)
    results = {}
    for algo in ("auto", "recurrent"):
        a = {n: x[n].clone().requires_grad_() for n in ("q", "k", "v", "g")}
        o, sT = lib.decay_linear_attention(a["q"], a["k"], a["v"], a["g"], scale=D ** -0.5, algo=algo)
        o.backward(x["do"])
        fo, fs = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], scale=D ** -0.5, algo=algo)
        # (the op asks for no ds0, and where the state's gradient is no result it is held in fewer bits)
        r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=D ** -0.5, algo=algo,
                            need_ds0=False)
        assert torch.equal(o, fo) and torch.equal(sT, fs)
        for n, t in a.items():
            assert torch.equal(t.grad, r["d" + n]), n
        results[algo] = o.detach()
    ref.check(results["recurrent"], want, ref.allowed(want, size, BF16, T, D, False), "o")
    assert not torch.equal(results["auto"], results["recurrent"])
