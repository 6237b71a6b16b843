"""Layer norm where lanes hold no elements, rows start anywhere and gradients arrive as views:
cases of their own beside test_layer_norm.py."""
import pytest
import torch

import linear_attention_rnn_wkv7_b200 as lib

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,D", [(F32, 3), (F32, 20), (F32, 100), (F32, 1020), (BF16, 3), (BF16, 72),
                                     (BF16, 200), (BF16, 1000)])
@pytest.mark.parametrize("value", [2.0 ** 70, -2.0 ** 70, 2.0 ** 100])
def test_huge_constant_rows_with_idle_lanes(cuda_device, dtype, D, value):
    """D times a power of two is exact in fp32, so the mean is the value and y is 0, whether or not
    every lane of a row's team holds elements (the mean's square is beyond fp32)."""
    x = torch.full((5, D), value, dtype=dtype, device="cuda")
    y, m, r = lib.wkv7_ln_fwd(x, eps=1e-5)
    assert bool((m == value).all()) and bool((y == 0).all())
    assert bool(((r * 1e-5 ** 0.5 - 1).abs() < 1e-6).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [7, 64, 1000])
def test_gradient_that_is_a_shifted_view(cuda_device, dtype, D):
    """An output joined behind an odd number of elements gets a dense gradient that is not 16-byte
    aligned."""
    gen = torch.Generator().manual_seed(D)
    x = torch.randn(9, D, generator=gen).to(dtype).cuda().requires_grad_()
    w, b = (torch.randn(D, generator=gen).cuda().to(dtype).requires_grad_() for _ in range(2))
    dy = torch.randn(9 * D + 1, generator=gen).to(dtype).cuda()
    y = lib.layer_norm(x, w, b)
    want = torch.autograd.grad(y, (x, w, b), dy[1:].clone().view(9, D), retain_graph=True)
    joined = torch.cat([torch.zeros(1, dtype=dtype, device="cuda"), y.flatten()])
    got = torch.autograd.grad(joined, (x, w, b), dy)
    for a, c in zip(got, want):
        assert torch.equal(a, c)


# D a multiple of the 16-byte group: only the statistics may lie anywhere; else every tensor
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [1, 7, 129, 1021, 8193, 64, 4096])
def test_rows_of_a_larger_tensor(cuda_device, dtype, D):
    """Rows from the second on: dense, and aligned to an element where a row is no multiple of 16
    bytes.  They give what the same rows in a tensor of their own give."""
    gen = torch.Generator().manual_seed(D)
    x, dy = (torch.randn(6, D, generator=gen).to(dtype).cuda() for _ in range(2))
    p = torch.randn(2, 1 + D if D % 8 else D, generator=gen).to(dtype).cuda()
    w, b = (p.flatten()[1:1 + D], p.flatten()[1 + D:1 + 2 * D]) if D % 8 else (p[0], p[1])
    want, wm, wr = lib.wkv7_ln_fwd(x[1:].clone(), w.clone(), b.clone())
    out = torch.empty_like(x)
    y, m, r = lib.wkv7_ln_fwd(x[1:], w, b, y=out[1:])
    assert torch.equal(y, want) and torch.equal(m, wm) and torch.equal(r, wr)
    wg = lib.wkv7_ln_bwd(x[1:].clone(), dy[1:].clone(), wm, wr, w.clone())
    mean, rstd = (torch.cat([t[:1], t]) for t in (wm, wr))
    g = lib.wkv7_ln_bwd(x[1:], dy[1:], mean[1:], rstd[1:], w)
    for n in g:
        assert torch.equal(g[n], wg[n]), n
