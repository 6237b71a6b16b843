"""The failure path of the decay linear attention's tensor-core kernel, made to run without any fault.

Every wait of that kernel is bounded.  A thread that gives up sets a flag that ends its block's other
waits; the block waits (bounded) for its copies and MMAs in flight, frees its tensor memory
and returns, and WKV7_ERR_DEVICE_TIMEOUT is reported once.  The test hook shortens the next call's
limits: of the wait for a state that the block before hands on (there for certain where a sequence
is longer than a block's run), and of all waits, so that roles give up anywhere, with copies
and MMAs behind them."""
import pytest
import torch

import la_walk
import linear_attention_rnn_wkv7_b200 as lib
from linear_attention_rnn_wkv7_b200 import build as lib_build
from linear_attention_rnn_wkv7_b200.wkv7 import ERR_DEVICE_TIMEOUT, ERR_INVALID_ARG, OK

BF16 = torch.bfloat16


def chain(H):
    """Offsets of 45 sequences, one of them many runs long."""
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(1, 60, (44,), generator=gen).tolist()
    lens.insert(20, 9000)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def problem(B, T, H, D, N, seed):
    gen = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, T, H, D, generator=gen).to(BF16).cuda() for n in ("q", "k", "v", "do")}
    x["g"] = -torch.rand(B, T, H, generator=gen).to(BF16).cuda()
    x["s0"] = torch.randn(N, H, D, D, generator=gen).cuda()
    return x


def run(x, cu=None):
    o, s = lib.wkv7_la_fwd(x["q"], x["k"], x["v"], x["g"], s0=x["s0"], cu_seqlens=cu)
    return {"o": o, "sT": s}


def run_bwd(x, cu=None):
    return lib.wkv7_la_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], s0=x["s0"], dsT=x["s0"], cu_seqlens=cu)


def test_hook_arguments():
    lib_build.build()
    clib = lib.library()
    assert clib.wkv7_test_hurry_next_la(-2, 0) == ERR_INVALID_ARG
    assert clib.wkv7_test_hurry_next_la(1000000001, 0) == ERR_INVALID_ARG
    assert clib.wkv7_test_hurry_next_la(1000000000, 1) == OK
    assert clib.wkv7_test_hurry_next_la(-1, 0) == OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_handoff_that_does_not_come(cuda_device, D):
    """Blocks in the middle of the long sequence look for a state that is some microseconds away and give
    up.  A sequence none of whose blocks waits for another is right, bit for bit."""
    H, cu = 4, chain(4)
    N, T = len(cu) - 1, cu[-1]
    x, cu_t = problem(1, T, H, D, N, D), torch.tensor(cu, dtype=torch.int32, device="cuda")
    for call, backward in ((run, False), (run_bwd, True)):
        want = call(x, cu_t)
        assert lib.wkv7_get_last_error() == OK
        assert lib.library().wkv7_test_hurry_next_la(20000000, 1) == OK
        got = call(x, cu_t)
        assert lib.wkv7_get_last_error() == ERR_DEVICE_TIMEOUT
        assert lib.wkv7_get_last_error() == OK               # cleared once read
        safe = torch.ones(N, H, dtype=torch.bool)
        waits = 0
        for against in ([False, True] if backward else [False]):
            pieces, _ = la_walk.walk(lib.library(), T, H, N, cu, D=D, backward=against)
            for rows in pieces:
                if all(r[4] for r in rows):
                    continue
                waits += 1
                for n, h, *_ in rows:
                    safe[n, h] = False
        assert waits > 8 and int(safe.sum()) > N          # both kinds are there
        for n in range(N):
            for h in range(H):
                if not safe[n, h]:
                    continue
                for name in got:
                    a, b = got[name], want[name]
                    if name in ("sT", "ds0"):
                        assert torch.equal(a[n, h], b[n, h]), (name, n, h)
                    else:
                        assert torch.equal(a[0, cu[n]:cu[n + 1], h], b[0, cu[n]:cu[n + 1], h]), (name, n, h)
        again = call(x, cu_t)                                # the hook was taken by that call
        for name in want:
            assert torch.equal(again[name], want[name]), name
        assert lib.wkv7_get_last_error() == OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["whole sequences", "runs", "segments", "one long of many"])
def test_waits_that_run_out_anywhere(cuda_device, D, kind):
    """All waits cut short, from none to 20 us: whatever gave up, the call returns, the status is this one
    or none, and the next call is exact."""
    cu = None
    if kind == "one long of many":
        cu = chain(4)
        x = problem(1, cu[-1], 4, D, len(cu) - 1, D)
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    else:
        B, T, H = {"whole sequences": (2, 900, 64), "runs": (40, 300, 4), "segments": (1, 6000, 2)}[kind]
        x = problem(B, T, H, D, B, D)
    seen = set()
    for call in (run, run_bwd):
        want = call(x, cu)
        assert lib.wkv7_get_last_error() == OK
        for wait in (0, 200, 1000, 3000, 20000):
            assert lib.library().wkv7_test_hurry_next_la(wait, int(wait == 0)) == OK
            call(x, cu)
            status = lib.wkv7_get_last_error()
            assert status in (OK, ERR_DEVICE_TIMEOUT)
            seen.add(status)
            again = call(x, cu)
            for name in want:
                assert torch.equal(again[name], want[name]), (name, wait)
            assert lib.wkv7_get_last_error() == OK
    # (wait = 0: a handoff that is hundreds of microseconds away)
    assert kind != "one long of many" or ERR_DEVICE_TIMEOUT in seen
