"""The shared memory that the expert layer's second product asks for covers all that a CTA
touches, for every number of tokens, slots and CTAs per tile."""
import ctypes

import pytest

ROW = 64 * 4          # bytes of a staged row: a tile's columns in fp32
STAGE_AT = 8192       # the rows follow the slots' tables
STAGE_ROWS = 192      # staged at a time
ROUND = 1023          # the start is rounded up to 1024 bytes


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("G", [-1, 32, 64, 96, 128])
def test_second_product_asks_for_what_it_touches(libwq, bits, G):
    L, used = libwq.lib(), ctypes.c_size_t()
    short = []
    for T in range(1, 65):
        for k in range(1, 17):
            for cluster in range(1, 9):
                asked = L.wq_moe_selftest_smem(T, k, 384, bits, G, cluster, ctypes.byref(used))
                assert 0 < asked <= 112 * 1024 and used.value > 0   # two CTAs per SM
                end = used.value
                if T > 16:   # the rows of a CTA's tokens, in portions of whole tokens
                    rows = min(STAGE_ROWS // k, -(-T // cluster)) * k
                    end = max(end, ROUND + STAGE_AT + rows * ROW)
                if asked < end:
                    short.append((T, k, cluster, asked, end))
    assert not short, f"{len(short)} launches ask for less than they touch, first {short[0]}"


def test_refuses_what_the_layer_refuses(libwq):
    L, used = libwq.lib(), ctypes.c_size_t()
    for a in ((0, 1, 64, 4, 32, 1), (65, 1, 64, 4, 32, 1), (1, 17, 64, 4, 32, 1), (1, 1, 0, 4, 32, 1),
              (1, 1, 64, 3, 32, 1), (1, 1, 64, 4, 16, 1), (1, 1, 64, 4, 0, 1), (1, 1, 64, 4, 32, 9)):
        assert L.wq_moe_selftest_smem(*a, ctypes.byref(used)) == 0
    assert L.wq_moe_selftest_smem(1, 1, 64, 4, 32, 1, None) == 0
