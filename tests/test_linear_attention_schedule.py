"""Which blocks of the decay linear attention work on which tokens, walked on the CPU by the kernels'
own code: every token of every sequence once, nothing else, and an end for any offsets."""
import ctypes

import pytest
import torch

import linear_attention_rnn_wkv7_b200 as lib
from linear_attention_rnn_wkv7_b200 import build as lib_build
from linear_attention_rnn_wkv7_b200.wkv7 import (ERR_DEVICE_BAD_SEQLENS, ERR_INVALID_ARG,
                                                 ERR_UNSUPPORTED, OK)
from la_walk import walk

F32, BF16 = 1, 0


@pytest.fixture(scope="module")
def clib():
    lib_build.build()
    return lib.library()


def check_cover(pieces, H, lens):
    seen = {}
    for rows in pieces:
        for n, h, tb, te, begins, ends in rows:
            assert 0 <= n < len(lens) and 0 <= h < H, (n, h)
            assert 0 <= tb <= te <= lens[n], (n, tb, te)
            seen.setdefault((n, h), []).append((tb, te, begins, ends))
    assert len(seen) == len(lens) * H          # an empty sequence has a piece too (its state)
    for (n, h), parts in seen.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == lens[n], (n, h, parts)
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:])), (n, h, parts)
        assert sum(p[2] for p in parts) == 1 and sum(p[3] for p in parts) == 1, (n, h, parts)


def lengths(seed, n, most):
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, most, (n,), generator=gen).tolist()
    lens[n // 2] = 0
    return lens


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,most", [(1, 3, 5000), (3, 4, 700), (8, 32, 300), (50, 4, 260)])
def test_packed_cover(clib, backward, dtype, N, H, most):
    """Segments (few pairs) and runs, tensor cores and the recurrent kernel; also with rows behind
    the last sequence."""
    lens = lengths(N, N, most) if N > 1 else [most]
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    for tail in (0, 1000):
        pieces, skipped = walk(clib, cu[-1] + tail, H, N, cu, dtype=dtype, backward=backward)
        assert not skipped
        check_cover(pieces, H, lens)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,T", [(1, 3, 5000), (2, 64, 300), (40, 4, 300), (148, 1, 129), (5, 32, 1),
                                   (4, 50, 1000)])
def test_unpacked_cover(clib, backward, dtype, N, H, T):
    pieces, _ = walk(clib, T, H, N, dtype=dtype, backward=backward)
    check_cover(pieces, H, [T] * N)


BAD = [[200, 250, 300, 340, 400, 410, 600, 777, 900],    # 8 sequences behind 200 rows
       [1, 250, 300, 340, 400, 410, 600, 777, 900],
       [128, 128, 128, 128, 128, 128, 128, 128, 128],
       [899, 899, 899, 899, 899, 899, 899, 899, 900]]


@pytest.mark.parametrize("cu", BAD)
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [2, 32])
def test_offsets_that_do_not_begin_at_0(clib, cu, backward, dtype, H):
    """They are reported and the call is skipped (cu_seqlens[0] = 0, include/wkv7.h); and even the
    walk that is then never begun has an end and touches the sequences' tokens alone."""
    pieces, skipped = walk(clib, 900, H, 8, cu, dtype=dtype, backward=backward)
    assert skipped
    check_cover(pieces, H, [b - a for a, b in zip(cu, cu[1:])])


@pytest.mark.parametrize("cu,bad", [([0, 5, 3, 9], True), ([0, 5, 10, 901], True), ([-1, 5, 10, 20], True),
                                    ([0, 0, 0, 0], False), ([0, 900, 900, 900], False)])
def test_order_and_range(clib, cu, bad):
    host, n = (ctypes.c_int32 * 4)(*cu), ctypes.c_int()
    skipped, one = ctypes.c_int(), (ctypes.c_int32 * 6)()
    assert clib.wkv7_test_la_pieces(1, 900, 2, 64, host, 3, BF16, 0, 0, one, 0, ctypes.byref(n),
                                    ctypes.byref(n), ctypes.byref(skipped)) == OK
    assert bool(skipped.value) == bad


P = 0x7f0000000000


@pytest.mark.parametrize("kw,status", [
    (dict(x0=P + 8), ERR_INVALID_ARG), (dict(x2=P + 2), ERR_INVALID_ARG), (dict(s=P + 1), ERR_INVALID_ARG),
    (dict(cu=0), ERR_INVALID_ARG), (dict(cu=P + 2), ERR_INVALID_ARG), (dict(T=-1), ERR_INVALID_ARG),
    (dict(H=0), ERR_INVALID_ARG), (dict(N=-1), ERR_INVALID_ARG), (dict(layout=2), ERR_INVALID_ARG),
    (dict(dtype=2), ERR_INVALID_ARG), (dict(K=96), ERR_UNSUPPORTED), (dict(T=0), OK),
])
def test_zero_tail_refuses(clib, kw, status):
    a = dict(x0=P, x1=P + (1 << 20), x2=P + (2 << 20), s=P + 4096, T=64, H=4, K=64, cu=P + 64, N=2,
             layout=0, dtype=0)
    a.update(kw)
    assert clib.wkv7_la_zero_tail(*(ctypes.c_void_p(a[n]) for n in ("x0", "x1", "x2", "s")), a["T"],
                                  a["H"], a["K"], ctypes.c_void_p(a["cu"]), a["N"], a["layout"],
                                  a["dtype"], None) == status


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("H", [2, 32])
@pytest.mark.parametrize("cu", BAD[:2])
def test_offsets_that_do_not_begin_at_0_skip_the_call(cuda_device, dtype, D, H, cu):
    gen = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(1, 900, H, D, generator=gen).to(dtype).cuda() for _ in range(4))
    g = -torch.rand(1, 900, H, generator=gen).to(dtype).cuda()
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o = torch.full_like(v, 3.0)
    sT = torch.full((8, H, D, D), 3.0, device="cuda")
    for algo in ("auto", "recurrent"):
        lib.wkv7_la_fwd(q, k, v, g, cu_seqlens=cu_t, o=o, sT=sT, algo=algo)
        assert lib.wkv7_get_last_error() == ERR_DEVICE_BAD_SEQLENS
        assert bool((o == 3.0).all()) and bool((sT == 3.0).all())
        for decay in (g, g[0, 0].contiguous()):
            lib.wkv7_la_bwd(q, k, v, decay, do, cu_seqlens=cu_t, algo=algo)
            assert lib.wkv7_get_last_error() == ERR_DEVICE_BAD_SEQLENS
    assert lib.wkv7_get_last_error() == OK
