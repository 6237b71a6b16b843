"""The blocks' work of the decay linear attention, walked on the CPU by the kernels' own code."""
import ctypes

from linear_attention_rnn_wkv7_b200.wkv7 import OK


def walk(clib, T, H, N, cu=None, D=64, dtype=0, backward=False):
    """Every block's pieces, and whether the kernels skip the call."""
    host = None if cu is None else (ctypes.c_int32 * len(cu))(*cu)
    # no walk has more pieces than the problem has (segment, head) pairs; segments have 32 tokens or more
    most = (T // 32 + 2) * N * H + 1
    room = (ctypes.c_int32 * (6 * most))()
    count, blocks, skipped = ctypes.c_int(), ctypes.c_int(1), ctypes.c_int()
    pieces, block = [], 0
    while block < blocks.value:
        assert clib.wkv7_test_la_pieces(1 if cu else N, T, H, D, host, N, dtype, int(backward), block,
                                        room, most, ctypes.byref(count), ctypes.byref(blocks),
                                        ctypes.byref(skipped)) == OK
        assert count.value < most, f"block {block} finds no end"
        pieces.append([tuple(room[6 * i:6 * i + 6]) for i in range(count.value)])
        block += 1
    return pieces, bool(skipped.value)
