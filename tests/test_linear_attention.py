"""The decay linear attention against its definition in fp64 (la_util.py), on the GPU; its
refusals and its reference's gradients on the CPU.  Tolerances: la_util.allowed."""
import ctypes

import pytest
import torch

import la_util as ref
import linear_attention_rnn_wkv7_b200 as lib
from linear_attention_rnn_wkv7_b200 import build as lib_build
from linear_attention_rnn_wkv7_b200.wkv7 import (ERR_DEVICE_BAD_SEQLENS, ERR_INVALID_ARG,
                                                 ERR_UNSUPPORTED, OK)

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(B, T, H, D, dtype, seed, gate="token", head_first=False, N=None, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    lead = (B, H, T) if head_first else (B, T, H)
    x = {n: torch.randn(*lead, D, generator=gen) for n in ("q", "k", "v", "do")}
    x["k"] = x["k"] / x["k"].norm(dim=-1, keepdim=True).clamp(min=1e-6)
    if gate == "token":
        x["g"] = -torch.rand(*lead, generator=gen) ** 4 * 3.0     # most weak, some strong
    else:
        x["g"] = torch.log1p(-torch.exp2(-5 + 3 * torch.rand(H, generator=gen)))
    x = {n: t.to(dtype) for n, t in x.items()}
    N = B if N is None else N
    x["s0"] = 0.3 * torch.randn(N, H, D, D, generator=gen)
    x["dsT"] = 0.3 * torch.randn(N, H, D, D, generator=gen)
    x["mask"] = (torch.rand(B, T, generator=gen) > 0.2).to(torch.uint8)
    return {n: t.to(device) for n, t in x.items()}


def tensor_cores(dtype, D, algo):
    return dtype == BF16 and D <= 128 and algo != "recurrent"


def compare_fwd(x, dtype, D, algo="auto", s0=True, mask=False, cu=None, head_first=False,
                scale=0.125, length=None):
    s0 = x["s0"] if s0 else None
    mask = x["mask"] if mask else None
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, sT = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=s0, mask=mask, cu_seqlens=cu_t,
                            scale=scale, algo=algo, head_first=head_first)
    args = (x["q"], x["k"], x["v"], x["g"], s0, mask, cu, scale, head_first)
    ro, rs = ref.forward(*args)
    mo, ms = ref.forward(*args, absolute=True)
    T = length or x["q"].shape[2 if head_first else 1]
    tc = tensor_cores(dtype, D, algo)
    eo = ref.check(o, ro, ref.allowed(ro, mo, dtype, T, D, tc), "o")
    es = ref.check(sT, rs, ref.allowed(rs, ms, dtype, T, D, tc, state=True), "sT")
    # the terms' roundings are independent: in the 2-norm far below the bound of each
    assert eo <= (5e-3 if dtype == BF16 else 2e-6) and es <= 5e-6, (eo, es)
    assert lib.wkv7_get_last_error() == OK


def compare_bwd(x, dtype, D, algo="auto", s0=True, mask=False, cu=None, head_first=False,
                scale=0.125, dsT=True):
    s0 = x["s0"] if s0 else None
    mask = x["mask"] if mask else None
    dsT = x["dsT"] if dsT else None
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=s0, mask=mask, dsT=dsT,
                          cu_seqlens=cu_t, scale=scale, algo=algo, head_first=head_first)
    args = (x["q"], x["k"], x["v"], x["g"], x["do"], s0, mask, dsT, cu, scale, head_first)
    r = ref.backward(*args)
    m = ref.backward(*args, absolute=True, chunk_sums=True)
    T = x["q"].shape[2 if head_first else 1]
    tc = tensor_cores(dtype, D, algo)
    for n in ("dq", "dk", "dv", "dg", "ds0"):
        tol = ref.allowed(r[n], m[n], dtype, T + 128, D, tc, state=n == "ds0")
        if n == "dg":
            # the products of q and dq, k and dk and of the two states: one more rounding
            # each of the kept state and the state's copy
            tol = tol + (ref.U_BF16 if tc else 0.0) * m[n] * 2
        e = ref.check(got[n], r[n], tol, n)
        lim = (5e-6 if n == "ds0" else 6e-3) if dtype == BF16 else 5e-6
        assert e <= lim, (n, e)
    assert lib.wkv7_get_last_error() == OK


# ------------------------------------------------------------------------- CPU: reference
def test_reference_gradients_by_differences():
    x = make(1, 5, 2, 3, torch.float64, 1, device="cpu")
    mask = torch.tensor([[1, 0, 1, 1, 1]], dtype=torch.uint8)
    cu = [0, 2, 2, 5]
    x["s0"] = torch.randn(3, 2, 3, 3, dtype=torch.float64)
    dsT = torch.randn(3, 2, 3, 3, dtype=torch.float64)

    def loss(q, k, v, g, s0):
        o, sT = ref.forward(q, k, v, g, s0, mask, cu, 0.7)
        return (o * x["do"]).sum() + (sT * dsT).sum()

    names = ("q", "k", "v", "g", "s0")
    r = ref.backward(x["q"], x["k"], x["v"], x["g"], x["do"], x["s0"], mask, dsT, cu, 0.7)
    for n in names:
        grad = r["ds0" if n == "s0" else "d" + n]
        flat, gf = x[n].reshape(-1), grad.reshape(-1)
        for i in range(0, flat.numel(), 7):
            d = torch.zeros_like(flat)
            d[i] = 1e-5
            d = d.reshape(x[n].shape)
            up = loss(*(x[m] + d if m == n else x[m] for m in names))
            dn = loss(*(x[m] - d if m == n else x[m] for m in names))
            # central differences: error of order 1e-10 from the step, 1e-11 from rounding
            assert abs(float(up - dn) / 2e-5 - float(gf[i])) < 1e-7, (n, i)


# -------------------------------------------------------------------------- CPU: refusals
P = 0x7f0000000000


@pytest.fixture(scope="module")
def clib():
    lib_build.build()
    return lib.library()


def p(x):
    return ctypes.c_void_p(x)


def fwd_args(**kw):
    a = dict(q=P, k=P + 4096, v=P + 8192, g=P + 64, gh=0, s0=0, mask=0, o=P + 16384, sT=0, B=2,
             T=64, H=4, K=64, V=64, cu=0, N=2, scale=1.0, layout=0, dtype=0, algo=0, ws=0, wsb=0)
    a.update(kw)
    return [p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), a["gh"], p(a["s0"]), p(a["mask"]),
            p(a["o"]), p(a["sT"]), a["B"], a["T"], a["H"], a["K"], a["V"], p(a["cu"]), a["N"],
            a["scale"], a["layout"], a["dtype"], a["algo"], p(a["ws"]), a["wsb"], None]


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), ERR_INVALID_ARG), (dict(k=P + 2), ERR_INVALID_ARG), (dict(g=0), ERR_INVALID_ARG),
    (dict(g=P + 1), ERR_INVALID_ARG), (dict(o=P), ERR_INVALID_ARG), (dict(sT=P + 4),
                                                                     ERR_INVALID_ARG),
    (dict(N=3), ERR_INVALID_ARG), (dict(cu=P), ERR_INVALID_ARG),
    (dict(cu=P + 2, B=1, N=5), ERR_INVALID_ARG), (dict(B=-1, N=-1), ERR_INVALID_ARG),
    (dict(H=0), ERR_INVALID_ARG), (dict(layout=2), ERR_INVALID_ARG),
    (dict(dtype=3), ERR_INVALID_ARG), (dict(algo=7), ERR_INVALID_ARG),
    (dict(scale=float("nan")), ERR_INVALID_ARG), (dict(scale=float("inf")), ERR_INVALID_ARG),
    (dict(K=64, V=128), ERR_UNSUPPORTED), (dict(K=96, V=96), ERR_UNSUPPORTED),
    (dict(dtype=1, algo=2), ERR_UNSUPPORTED), (dict(K=256, V=256, algo=2), ERR_UNSUPPORTED),
    (dict(B=1 << 20, N=1 << 20, T=1 << 20), ERR_UNSUPPORTED),
    # one long sequence is cut into segments and needs the workspace
    (dict(B=1, N=1, H=1, T=8192), ERR_INVALID_ARG),
    (dict(B=1, N=1, H=1, T=8192, ws=P + 3, wsb=1 << 40), ERR_INVALID_ARG),
])
def test_fwd_refuses(clib, kw, status):
    assert clib.wkv7_la_fwd(*fwd_args(**kw)) == status


def bwd_args(**kw):
    a = dict(q=P, k=P + 4096, v=P + 8192, g=P + 64, gh=0, s0=0, mask=0, do=P + (1 << 20), dsT=0,
             dq=P + (2 << 20), dk=P + (3 << 20), dv=P + (4 << 20), dg=P + (5 << 20), ds0=0, B=2,
             T=64, H=4, K=64, V=64, cu=0, N=2, scale=1.0, layout=0, dtype=0, algo=0, ws=P,
             wsb=1 << 40)
    a.update(kw)
    return [p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), a["gh"], p(a["s0"]), p(a["mask"]),
            p(a["do"]), p(a["dsT"]), p(a["dq"]), p(a["dk"]), p(a["dv"]), p(a["dg"]), p(a["ds0"]),
            a["B"], a["T"], a["H"], a["K"], a["V"], p(a["cu"]), a["N"], a["scale"], a["layout"],
            a["dtype"], a["algo"], p(a["ws"]), a["wsb"], None]


@pytest.mark.parametrize("kw,status", [
    (dict(do=0), ERR_INVALID_ARG), (dict(dq=P), ERR_INVALID_ARG), (dict(dk=P + (2 << 20)),
                                                                   ERR_INVALID_ARG),
    (dict(dv=0), ERR_INVALID_ARG), (dict(dg=P + 64), ERR_INVALID_ARG),
    (dict(ds0=P + 4), ERR_INVALID_ARG), (dict(ds0=P + 32, dsT=P + 32), ERR_INVALID_ARG),
    (dict(ws=0), ERR_INVALID_ARG), (dict(wsb=16), ERR_INVALID_ARG),
    (dict(K=32, V=32), ERR_UNSUPPORTED), (dict(dtype=1, algo=2), ERR_UNSUPPORTED),
    (dict(N=1), ERR_INVALID_ARG), (dict(scale=float("nan")), ERR_INVALID_ARG),
])
def test_bwd_refuses(clib, kw, status):
    assert clib.wkv7_la_bwd(*bwd_args(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), ERR_INVALID_ARG), (dict(state=P + 8), ERR_INVALID_ARG),
    (dict(o=P), ERR_INVALID_ARG), (dict(K=64, V=128), ERR_UNSUPPORTED),
    (dict(H=0), ERR_INVALID_ARG), (dict(out=0), ERR_INVALID_ARG),
    (dict(scale=float("inf")), ERR_INVALID_ARG),
])
def test_step_refuses(clib, kw, status):
    a = dict(q=P, k=P + 4096, v=P + 8192, g=P + 64, state=P + (1 << 20), out=P + (1 << 20),
             o=P + 16384, B=2, H=4, K=64, V=64, scale=1.0, dtype=0)
    a.update(kw)
    assert clib.wkv7_la_step(p(a["q"]), p(a["k"]), p(a["v"]), p(a["g"]), 0, p(a["state"]),
                             p(a["out"]), p(a["o"]), a["B"], a["H"], a["K"], a["V"], a["scale"],
                             a["dtype"], None) == status


def test_workspace_queries(clib):
    q = lib.wkv7_la_workspace_bytes
    assert q(8, 4096, 64) == 0                     # sequences fill the GPU: nothing is cut
    assert q(5, 4096, 32) > 0                      # states handed from block to block
    assert q(1, 16384, 4) > 0 and q(1, 16384, 4, 128, 128) > q(1, 16384, 4)
    assert q(1, 100, 1) == 0 and q(1, 0, 1) == 0
    assert q(2, 100, 4, backward=True) > 0
    assert q(1, 100, 4, 64, 128) == 0              # unsupported
    assert q(2, 100, 4, N=3) == 0                  # N must be B unless packed


def test_binding_refuses_cpu_and_wrong_tensors():
    x = make(1, 4, 2, 64, F32, 0, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"])
    with pytest.raises(ValueError, match="CUDA"):
        lib.decay_linear_attention(x["q"], x["k"], x["v"], x["g"])
    with pytest.raises(ValueError, match="CUDA"):
        lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"])
    with pytest.raises(ValueError, match="CUDA"):
        lib.wkv7_la_step(x["q"][0], x["k"][0], x["v"][0], x["g"][0], x["s0"])


# ---------------------------------------------------------------------------- GPU: forward
@gpu
@pytest.mark.parametrize("algo", ["recurrent", "auto"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 17, 128, 300])
def test_fwd(cuda_device, algo, dtype, D, T):
    x = make(2, T, 3, D, dtype, T + D)
    compare_fwd(x, dtype, D, algo)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128), (BF16, 256)])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("head_first", [False, True])
def test_fwd_masked(cuda_device, dtype, D, gate, head_first):
    x = make(3, 261, 2, D, dtype, 5, gate, head_first)
    x["mask"][1] = 0                      # a row with no live token
    x["mask"][2, 128:] = 0                # a chunk without one
    # what masked tokens hold must not matter
    for n in ("k", "v"):
        t = x[n].transpose(1, 2) if head_first else x[n]
        t[x["mask"] == 0] = float("nan")
    if gate == "token":
        t = x["g"].transpose(1, 2) if head_first else x["g"]
        t[x["mask"] == 0] = float("inf")
    compare_fwd(x, dtype, D, mask=True, head_first=head_first)
    compare_fwd(x, dtype, D, mask=True, head_first=head_first, s0=False, algo="recurrent")


CU = [0, 0, 1, 128, 257, 257, 600, 611]


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 128), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("head_first", [False, True])
def test_fwd_packed(cuda_device, dtype, D, head_first):
    x = make(1, CU[-1], 3, D, dtype, 7, head_first=head_first, N=len(CU) - 1)
    compare_fwd(x, dtype, D, cu=CU, head_first=head_first)
    compare_fwd(x, dtype, D, cu=CU, head_first=head_first, mask=True, s0=False)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 256), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_fwd_cut_into_segments(cuda_device, dtype, D, gate):
    assert lib.wkv7_la_workspace_bytes(1, 1500, 2, D, D, dtype=dtype) > 0
    x = make(1, 1500, 2, D, dtype, 11, gate)
    compare_fwd(x, dtype, D)
    compare_fwd(x, dtype, D, mask=True)
    x = make(1, 1500, 2, D, dtype, 12, gate, N=3)
    compare_fwd(x, dtype, D, cu=[0, 3, 1200, 1500])


def many_sequences(D, seed, packed, head_first=False):
    """More (sequence, head) pairs than SMs, so that sequences are cut between blocks: of one
    length, or packed with lengths from 0 to more than a block's share."""
    if not packed:
        return make(40, 300, 4, D, BF16, seed, head_first=head_first), None
    gen = torch.Generator().manual_seed(seed)
    lens = [0, 1, 128, 700, 0] + torch.randint(0, 60, (45,), generator=gen).tolist() + [257, 0]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return make(1, cu[-1], 4, D, BF16, seed, head_first=head_first, N=len(lens)), cu


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("packed,head_first", [(False, False), (True, False), (True, True)])
def test_many_sequences(cuda_device, D, packed, head_first):
    x, cu = many_sequences(D, 71, packed, head_first)
    compare_fwd(x, BF16, D, cu=cu, head_first=head_first)
    compare_bwd(x, BF16, D, cu=cu, head_first=head_first, mask=True)


@gpu
def test_many_sequences_repeat_and_replay(cuda_device):
    """States handed between blocks: the same bits from call to call and from a replayed graph."""
    x, cu = many_sequences(64, 73, True)
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    call = lambda: (lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], cu_seqlens=cu),  # noqa: E731
                    lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu))
    (o, s), b = call()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        (o2, s2), b2 = call()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(s, s2)
        for n in b:
            assert torch.equal(b[n], b2[n]), n
    assert lib.wkv7_get_last_error() == OK


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_fwd_strong_decays_and_resets(cuda_device, dtype, D):
    x = make(1, 400, 2, D, dtype, 13)
    x["g"][:, 100:220] = -50.0            # e^{-50} a token: nothing survives
    x["g"][:, 300] = float("-inf")        # a reset
    x["g"][:, 301] = 0.0
    compare_fwd(x, dtype, D)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_fwd_leaves_other_rows_and_sequences_alone(cuda_device, dtype, D):
    """Rows behind the last sequence keep what they hold, and what other sequences' rows hold
    (NaN) does not reach a sequence through a shared tile."""
    cu, T = [0, 70, 200], 333
    x = make(1, T, 2, D, dtype, 17, N=2)
    for n in ("q", "k", "v", "g", "do"):
        x[n][:, 200:] = float("nan")
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(x["v"], 7.0)
    lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], cu_seqlens=cu_t, o=o)
    assert bool((o[:, 200:] == 7.0).all())
    first = o[:, :70].clone()
    assert bool(torch.isfinite(o[:, :200]).all())
    for n in ("q", "k", "v", "g"):
        x[n][:, 70:200] = float("nan")
    lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], cu_seqlens=cu_t, o=o)
    assert torch.equal(o[:, :70], first)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64)])
@pytest.mark.parametrize("cu", [[0, 70, 50, 100], [0, 50, 101], [-1, 50, 100]])
def test_bad_seqlens_skip_the_call(cuda_device, dtype, D, cu):
    x = make(1, 100, 2, D, dtype, 19, N=len(cu) - 1)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, sT = torch.full_like(x["v"], 3.0), torch.full_like(x["s0"], 3.0)
    lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu_t, o=o, sT=sT)
    assert lib.wkv7_get_last_error() == ERR_DEVICE_BAD_SEQLENS
    assert bool((o == 3.0).all()) and bool((sT == 3.0).all())
    assert lib.wkv7_get_last_error() == OK
    lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], cu_seqlens=cu_t)
    assert lib.wkv7_get_last_error() == ERR_DEVICE_BAD_SEQLENS


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_empty_problems(cuda_device, dtype):
    x = make(2, 0, 3, 64, dtype, 0)
    o, sT = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    assert o.shape == (2, 0, 3, 64) and torch.equal(sT, x["s0"])
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], dsT=x["dsT"])
    assert torch.equal(r["ds0"], x["dsT"])
    x = make(0, 5, 3, 64, dtype, 0, gate="head")
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"])
    assert torch.equal(r["dg"], torch.zeros_like(x["g"]))


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_state_in_place_and_runs_repeat(cuda_device, D):
    x = make(2, 200, 3, D, BF16, 23)
    o, sT = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
    s = x["s0"].clone()
    o2, s2 = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=s, sT=s)
    assert torch.equal(o, o2) and torch.equal(sT, s2) and s2.data_ptr() == s.data_ptr()


# --------------------------------------------------------------------------- GPU: backward
@gpu
@pytest.mark.parametrize("algo", ["recurrent", "auto"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 130])
def test_bwd(cuda_device, algo, dtype, D, T):
    x = make(2, T, 2, D, dtype, T + D)
    compare_bwd(x, dtype, D, algo)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("gate", ["token", "head"])
@pytest.mark.parametrize("head_first", [False, True])
def test_bwd_masked(cuda_device, dtype, D, gate, head_first):
    x = make(3, 261, 2, D, dtype, 29, gate, head_first)
    x["mask"][1] = 0
    x["mask"][2, 128:] = 0
    for n in ("k", "v"):
        t = x[n].transpose(1, 2) if head_first else x[n]
        t[x["mask"] == 0] = float("nan")
    compare_bwd(x, dtype, D, mask=True, head_first=head_first)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("head_first", [False, True])
def test_bwd_packed(cuda_device, dtype, D, head_first):
    x = make(1, CU[-1], 2, D, dtype, 31, head_first=head_first, N=len(CU) - 1)
    compare_bwd(x, dtype, D, cu=CU, head_first=head_first)
    compare_bwd(x, dtype, D, cu=CU, head_first=head_first, mask=True, s0=False, dsT=False)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_bwd_cut_into_segments(cuda_device, dtype, D, gate):
    x = make(1, 900, 2, D, dtype, 37, gate)
    compare_bwd(x, dtype, D)
    x = make(1, 900, 2, D, dtype, 38, gate, N=3)
    compare_bwd(x, dtype, D, cu=[0, 3, 800, 900], mask=True)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_bwd_strong_decays(cuda_device, dtype, D):
    x = make(1, 300, 2, D, dtype, 41)
    x["g"][:, 60:150] = -50.0
    x["g"][:, 200] = float("-inf")
    compare_bwd(x, dtype, D)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_bwd_by_differences(cuda_device, dtype, D):
    """A directional difference of the loss, from the fp64 form: the gradients' dot product with
    a direction, without the backward's formulas."""
    x = make(1, 150, 2, D, dtype, 43)
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], dsT=x["dsT"],
                        scale=0.125)
    gen = torch.Generator().manual_seed(1)
    names = ("q", "k", "v", "g", "s0")
    for n in names:
        d = torch.randn(x[n].shape, generator=gen).cuda().double()
        # along the gradient itself, so that the sum does not cancel
        grad = r["ds0" if n == "s0" else "d" + n].double()
        d = d * 0.1 + grad / grad.abs().max()

        def loss(h):
            y = {m: x[m].double() + (h * d if m == n else 0) for m in names}
            o, s = ref.forward(y["q"], y["k"], y["v"], y["g"], y["s0"], None, None, 0.125)
            return float((o * x["do"].double()).sum() + (s * x["dsT"].double()).sum())

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = float((grad * d).sum())
        # each gradient value is within a few half steps; the sum is dominated by grad^2
        assert abs(got - want) <= (0.02 if dtype == BF16 else 1e-4) * abs(want) + 1e-4, (n, got, want)


@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_bwd_repeats_bit_for_bit(cuda_device, dtype):
    x = make(2, 700, 4, 64, dtype, 47, "head")
    a = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"])
    b = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"])
    for n in a:
        assert torch.equal(a[n], b[n]), n


# ------------------------------------------------------------------------------- GPU: step
@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 5), (300, 5)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_step(cuda_device, dtype, D, B, H, gate):
    x = make(B, 1, H, D, dtype, D + B, gate)
    one = {n: x[n][:, 0].contiguous() for n in ("q", "k", "v")}
    g = x["g"][:, 0].contiguous() if gate == "token" else x["g"]
    out = torch.empty_like(x["s0"])
    o = lib.wkv7_la_step(one["q"], one["k"], one["v"], g, x["s0"], out_state=out, scale=0.5)
    args = (x["q"], x["k"], x["v"], x["g"], x["s0"], None, None, 0.5)
    ro, rs = ref.forward(*args)
    mo, ms = ref.forward(*args, absolute=True)
    ref.check(o, ro[:, 0], ref.allowed(ro, mo, dtype, 1, D, False)[:, 0], "o")
    ref.check(out, rs, ref.allowed(rs, ms, dtype, 1, D, False, state=True), "state")
    state = x["s0"].clone()
    o2 = lib.wkv7_la_step(one["q"], one["k"], one["v"], g, state, scale=0.5)
    assert torch.equal(o, o2) and torch.equal(state, out)


@gpu
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 64), (BF16, 128)])
def test_prompt_then_tokens(cuda_device, dtype, D):
    """A prompt through the sequence form, then tokens one by one on its state, as a server runs them."""
    x = make(2, 205, 3, D, dtype, 53)
    o, state = lib.wkv7_la_fwd(*(x[n][:, :200].contiguous() for n in "qkvg"), s0=x["s0"],
                               scale=0.125)
    ro, rs = ref.forward(x["q"], x["k"], x["v"], x["g"], x["s0"], None, None, 0.125)
    mo, ms = ref.forward(x["q"], x["k"], x["v"], x["g"], x["s0"], None, None, 0.125,
                         absolute=True)
    tc = tensor_cores(dtype, D, "auto")
    for t in range(200, 205):
        y = lib.wkv7_la_step(*(x[n][:, t].contiguous() for n in "qkvg"), state, scale=0.125)
        ref.check(y, ro[:, t], ref.allowed(ro, mo, dtype, 205, D, tc)[:, t], f"token {t}")
    ref.check(state, rs, ref.allowed(rs, ms, dtype, 205, D, tc, state=True), "state")


# ------------------------------------------------------------- GPU: streams, graphs, autograd
@gpu
def test_other_stream_and_graphs(cuda_device):
    """On a side stream, and two captured graphs replayed in turn, each with its own workspace."""
    xs = [make(1, 1500, 2, 64, BF16, s) for s in (61, 62)]
    want = [(lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"]),
             lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"])) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, s = lib.wkv7_la_fwd(*(xs[0][n] for n in "qkvg"), s0=xs[0]["s0"])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0][0][0]) and torch.equal(s, want[0][0][1])
    graphs, outs = [], []
    torch.cuda.synchronize()
    for x in xs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            f = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"])
            b = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"])
        graphs.append(gr)
        outs.append((f, b))
    for _ in range(2):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (f, b), (wf, wb) in zip(outs, want):
        assert torch.equal(f[0], wf[0]) and torch.equal(f[1], wf[1])
        for n in b:
            assert torch.equal(b[n], wb[n]), n
    assert lib.wkv7_get_last_error() == OK


@gpu
def test_autograd_op(cuda_device):
    x = make(2, 140, 2, 64, F32, 67, "head")
    leaves = {n: x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "s0")}
    o, sT = lib.decay_linear_attention(leaves["q"], leaves["k"], leaves["v"], leaves["g"],
                                       initial_state=leaves["s0"], scale=0.25)
    ((o * x["do"]).sum() + (sT * x["dsT"]).sum()).backward()
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], dsT=x["dsT"],
                        scale=0.25)
    for n, t in leaves.items():
        assert torch.equal(t.grad, r["ds0" if n == "s0" else "d" + n]), n
    # only the final state, no initial state, a view with another layout as a gradient
    q, k, v = (x[n].clone().requires_grad_() for n in "qkv")
    o, sT = lib.decay_linear_attention(q, k, v, x["g"], scale=0.25)
    (sT * x["dsT"]).sum().backward()
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], torch.zeros_like(x["do"]), dsT=x["dsT"],
                        scale=0.25)
    assert torch.equal(q.grad, r["dq"]) and torch.equal(k.grad, r["dk"])
    q.grad = None
    o, none = lib.decay_linear_attention(q, k, v, x["g"], output_final_state=False, scale=0.25)
    assert none is None
    do = x["do"].transpose(0, 1).contiguous().transpose(0, 1)   # not contiguous
    o.backward(do)
    r = lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=0.25)
    assert torch.equal(q.grad, r["dq"])
