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
