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
