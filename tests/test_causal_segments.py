"""How the convolution's backward pass cuts sequences into segments: the same choice as a search of every number of
groups, found without trying them all.  No GPU."""
import time

import pytest

from depthwise_convolution_gb300 import _lib

ROWS, LEAST, EDGE, SMS = 4, 8, 12, 152  # segments of a block, shortest segment, tokens an edge costs, SMs


def segment(B, T, C):
    """The rule: of all numbers of groups (until blocks are 1024 tokens and nine waves), the one whose waves of blocks
    take the fewest steps; the first of equals."""
    whole = C % 4 == 0
    slots, columns = SMS * (4 if whole else 8), B * ((C + 127) // 128 if whole else (C + 31) // 32)
    best, seg, groups = None, LEAST, 1
    while groups == 1 or groups * ROWS * LEAST < T + ROWS * LEAST:
        s = max(-(-T // (groups * ROWS)), LEAST)
        cost = -(-columns * groups // slots) * (s + EDGE)
        if best is None or cost < best:
            best, seg = cost, s
        if s <= 1024 and columns * groups > 8 * slots:
            break
        groups += 1
    return seg


def slices(B, T, C):
    return _lib.load().dwconv_causal_bwd_workspace_size(B, T, C, 4, _lib.BF16) // (5 * C * 4)


@pytest.mark.parametrize("B", [1, 2, 3, 7, 40, 700, 65535])
def test_the_choice_is_that_of_the_whole_search(B):
    for T in (1, 7, 8, 31, 32, 33, 127, 500, 777, 1024, 2048, 4097, 16383, 50000, 131072, 1 << 20, (1 << 24) - 1):
        for C in (1, 7, 30, 64, 96, 128, 136, 1000, 2304, 4096, 4097, 16384):
            if B * T * C <= 1 << 36:
                want = segment(B, T, C) * ROWS
                assert slices(B, T, C) == B * -(-T // want), (B, T, C)


def test_long_narrow_sequences_cost_no_more_to_plan():
    def cost(B, T, C):
        times = []
        for _ in range(5):
            start = time.perf_counter()
            for _ in range(20):
                slices(B, T, C)
            times.append(time.perf_counter() - start)
        return min(times)

    # every number of groups is some 4900 of them here, a hundred times the call itself
    assert cost(1, 1 << 22, 64) < 10 * cost(1, 100, 64)
