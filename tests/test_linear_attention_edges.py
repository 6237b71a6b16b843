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


# ------------------------------------------------- results of the state, and long sequences in 64 bits
def walk_forward(x, scale):
    """o and the final state in 64 bits, all sequences and heads at once."""
    S, g = x["s0"].double(), x["g"].double()
    B, T, H, _ = x["q"].shape
    g = g.expand(B, T, H) if g.dim() == 1 else g
    out = []
    for t in range(T):
        S = (torch.exp(g[:, t])[..., None, None] * S
             + x["k"][:, t].double()[..., :, None] * x["v"][:, t].double()[..., None, :])
        out.append(scale * (x["q"][:, t].double()[..., None, :] @ S)[..., 0, :])
    return torch.stack(out, 1), S


def random_problem(B, T, H, D, gate, seed):
    gen = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, T, H, D, generator=gen).to(BF16) for n in ("q", "k", "v", "do")}
    x["k"] = (x["k"].float() / x["k"].float().norm(dim=-1, keepdim=True)).to(BF16)
    if gate == "token":
        x["g"] = (-torch.rand(B, T, H, generator=gen) ** 4 * 3.0).to(BF16)
    else:                               # memories of 32 to 1024 tokens
        x["g"] = (-torch.exp2(-5 - 5 * torch.rand(H, generator=gen))).to(BF16)
    x["s0"] = 0.3 * torch.randn(B, H, D, D, generator=gen)
    x["dsT"] = 0.3 * torch.randn(B, H, D, D, generator=gen)
    return {n: t.cuda() for n, t in x.items()}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("B,T,H", [(1, 6000, 2), (2, 2000, 64), (40, 300, 4)])
def test_final_states_need_three_parts(cuda_device, D, gate, B, T, H):
    """sT (and ds0 below) of the tensor cores: a term's factors are two exponentials, within 2^-22 each,
    three products and a split in three bf16 parts, half a step of 2^-24 each, and as many
    decays of half a step as chunks in its memory (8 of these): 2 * 4 + 4 + 8 = 20 half steps if
    all fell together, 6e-8 * 20 = 1.2e-6.  They do not: 1e-6 in the 2-norm, which the update's
    operand in two parts (2^-16 of each term, 2.5e-6 here) does not reach."""
    x = random_problem(B, T, H, D, gate, B + T + D)
    o, sT = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], scale=D ** -0.5)
    want_o, want_s = walk_forward(x, D ** -0.5)
    assert float((sT.double() - want_s).norm() / want_s.norm()) <= 1e-6
    # o: its own rounding, the scores' and the state copy's (each 2^-8 / sqrt(3) / 1.4 at most)
    assert float((o.double() - want_o).norm() / want_o.norm()) <= 3e-3
    assert lib.wkv7_get_last_error() == OK


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("B,T,H", [(1, 4000, 2), (30, 260, 5)])
def test_gradients_of_long_sequences(cuda_device, D, gate, B, T, H):
    """ds0 as sT above; the others are bf16 with the same three roundings as o, dg with those of
    both products that it is the difference of.  A dg that is summed over batch and tokens may
    cancel (600 left of terms that add up to 1e5 in magnitude): each token's is off by at most three
    half steps of the magnitudes that its chunk adds (the scores, the state's copy, the kept
    state), so the sum by at most three of theirs, and its own rounding."""
    x = random_problem(B, T, H, D, gate, B + T + D)
    got = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], dsT=x["dsT"],
                          scale=D ** -0.5)
    args = (x["q"], x["k"], x["v"], x["g"], x["do"], x["s0"], None, x["dsT"], None, D ** -0.5)
    want = ref.backward(*args)
    for n, lim in (("dq", 3e-3), ("dk", 3e-3), ("dv", 3e-3), ("dg", 6e-3), ("ds0", 1e-6)):
        if n == "dg" and gate == "head":
            size = ref.backward(*args, absolute=True, chunk_sums=True)["dg"]
            ref.check(got[n], want[n], 3 * ref.U_BF16 * size * (1 + ref.U_BF16) + ref.U_BF16 * want[n].abs(), n)
            continue
        assert float((got[n].double() - want[n]).norm() / want[n].norm()) <= lim, n
    assert lib.wkv7_get_last_error() == OK


# ------------------------------------------------------------------------------ two calls at once
@pytest.mark.parametrize("kind", ["runs", "packed", "segments"])
def test_two_calls_at_once(cuda_device, kind):
    """Forward and backward on two streams at the same time, and rows behind the last sequence too: each
    call has its own workspace, and its blocks wait for its own blocks alone."""
    B, T, H, cu = {"runs": (40, 300, 4, None), "segments": (1, 3000, 2, None),
                   "packed": (1, 6000, 4, [0, 900, 900, 1000] + [1000 + 100 * i for i in range(1, 42)])}[kind]
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    N = B if cu is None else len(cu) - 1
    xs = []
    for seed in (1, 2):
        x = random_problem(B, T, H, 64, "token", seed)
        x["s0"] = torch.randn(N, H, 64, 64, generator=torch.Generator().manual_seed(seed)).cuda()
        xs.append(x)

    def call(x):
        o, s = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], cu_seqlens=cu_t)
        r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], cu_seqlens=cu_t)
        return {"o": o, "s": s, **r}

    want = [call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (x, st) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(st):
                got[i].append(call(x))
    torch.cuda.synchronize()
    for i in range(2):
        for one in got[i]:
            for n in one:
                assert torch.equal(one[n], want[i][n]), (n, i)
    assert lib.wkv7_get_last_error() == OK
    for st in streams:
        with torch.cuda.stream(st):
            assert lib.wkv7_get_last_error() == OK


# -------------------------------------------------- neighbours, states in place, offsets past 32 bits
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("H", [2, 40])
def test_gradients_do_not_see_other_sequences(cuda_device, dtype, D, H):
    """NaN in every row of the other sequences, which share tiles with this one, and behind the last."""
    gen = torch.Generator().manual_seed(D + H)
    cu, T = [0, 70, 200, 330, 331, 500], 560
    N = len(cu) - 1
    x = {n: torch.randn(1, T, H, D, generator=gen).to(dtype).cuda() for n in ("q", "k", "v", "do")}
    x["g"] = -torch.rand(1, T, H, generator=gen).to(dtype).cuda()
    s0, dsT = (torch.randn(N, H, D, D, generator=gen).cuda() for _ in range(2))
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call(y, a, b):
        return lib.wkv7_la_bwd(y["q"], y["k"], y["v"], y["g"], y["do"], s0=a, dsT=b, cu_seqlens=cu_t)

    want = call(x, s0, dsT)
    for n in range(N):
        y = {m: torch.full_like(t, float("nan")) for m, t in x.items()}
        a, b = torch.full_like(s0, float("nan")), torch.full_like(dsT, float("nan"))
        for m in y:
            y[m][:, cu[n]:cu[n + 1]] = x[m][:, cu[n]:cu[n + 1]]
        a[n], b[n] = s0[n], dsT[n]
        got = call(y, a, b)
        for m in ("dq", "dk", "dv", "dg"):
            assert torch.equal(got[m][:, cu[n]:cu[n + 1]], want[m][:, cu[n]:cu[n + 1]]), (m, n)
            assert bool((got[m][:, cu[-1]:] == 0).all()), m
        assert torch.equal(got["ds0"][n], want["ds0"][n]), n
    assert lib.wkv7_get_last_error() == OK


@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 256), (BF16, 64), (BF16, 128), (BF16, 256)])
@pytest.mark.parametrize("B,T,H", [(40, 300, 4), (1, 1500, 2), (2, 300, 64)])
def test_states_in_place(cuda_device, dtype, D, B, T, H):
    """sT over s0 where sequences are handed from block to block, cut into segments, or neither."""
    gen = torch.Generator().manual_seed(D + T)
    q, k, v = (torch.randn(B, T, H, D, generator=gen).to(dtype).cuda() for _ in range(3))
    g = -torch.rand(B, T, H, generator=gen).to(dtype).cuda() * 0.1
    s0 = torch.randn(B, H, D, D, generator=gen).cuda()
    o, sT = lib.wkv7_la_fwd(q, k, v, g, s0=s0)
    for _ in range(3):
        s = s0.clone()
        o2, s2 = lib.wkv7_la_fwd(q, k, v, g, s0=s, sT=s)
        assert s2.data_ptr() == s.data_ptr() and torch.equal(o, o2) and torch.equal(sT, s)


def test_more_elements_than_32_bits_count(cuda_device):
    """2.28e9 elements a tensor: the last batch row's results are those of a call of its own (cut
    differently: each is off by bf16's roundings of its terms), forward, backward and layer norm."""
    B, T, H, D = 34, 8192, 64, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = {n: torch.randn(B, T, H, D, device="cuda", generator=gen, dtype=BF16) for n in ("q", "k", "v", "do")}
    assert x["q"].numel() > 2 ** 31
    x["k"] *= D ** -0.5
    x["g"] = (-torch.rand(B, T, H, device="cuda", generator=gen) * 0.2).to(BF16)
    last = {n: t[-1:].clone() for n, t in x.items()}

    def rel(a, b):
        return float((a.double() - b.double()).norm() / b.double().norm())

    o, s = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], scale=D ** -0.5)
    lo, ls = lib.wkv7_la_fwd(last["q"], last["k"], last["v"], last["g"], scale=D ** -0.5)
    # two results that are each within 3e-3 (states 1e-6) of the definition
    assert rel(o[-1:], lo) <= 6e-3 and rel(s[-1:], ls) <= 2e-6
    y, m, r = lib.wkv7_ln_fwd(o)
    ly, lm, lr = lib.wkv7_ln_fwd(o[-1:].clone())
    assert torch.equal(y[-1:], ly) and torch.equal(m[-1:], lm) and torch.equal(r[-1:], lr)
    del y
    gx = lib.wkv7_ln_bwd(o, x["do"], m, r)["dx"]
    assert torch.equal(gx[-1:], lib.wkv7_ln_bwd(o[-1:].clone(), last["do"], lm, lr)["dx"])
    del gx, o
    b = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=D ** -0.5)
    lb = lib.wkv7_la_bwd(last["q"], last["k"], last["v"], last["g"], last["do"], scale=D ** -0.5)
    for n in ("dq", "dk", "dv", "dg", "ds0"):
        assert rel(b[n][-1:], lb[n]) <= (2e-6 if n == "ds0" else 1.2e-2 if n == "dg" else 6e-3), n
    assert lib.wkv7_get_last_error() == OK
