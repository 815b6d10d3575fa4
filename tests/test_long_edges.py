"""CPU checks beside test_gpu_long_edges: its cases of long lists are ones that the attention cuts into
pieces, and short ones are not; the oracle's appended codes stand for finite values."""
import numpy as np
import pytest

from oracle import blocks as ref8
from test_gpu_long_edges import CUT, pieces


@pytest.fixture(scope="module")
def jb():
    from gated_delta_rule_jetblock_amd import jetblock
    return jetblock


@pytest.mark.parametrize("case", CUT)
def test_long_lists_are_cut(jb, case):
    page, count = case[4:]
    for B, T, n, packed in ((6, 1, 6, False), (5, 17, 17, True), (5, 4, 17, True), (2, 3, 6, False), (1, 3, 3, True)):
        assert pieces(jb, B, T, n, *case, count + 2, packed) > 1
        assert pieces(jb, B, T, n, *case[:4], 16, 10, 12, packed) == 1


def test_largest_values_of_the_oracle():
    """The nearest code whose value is less than 2^128, under every scale that can pass it."""
    for e in range(246, 255):
        codes, scales = np.zeros((1, 1, 16, 4), np.uint8), np.full((1, 1, 1), e, np.uint8)
        fresh = np.array([[[np.finfo(np.float32).max, -1.9375 * 2.0 ** 127, 1.875 * 2.0 ** 127, np.inf]]])
        ref8.append(codes, scales, [0], 2, fresh)
        held = ref8.dequantise(codes, scales)[0, 0, 1]
        assert scales.ravel().tolist() == [max(e, 247)] and np.isnan(held[3])
        assert (np.abs(held[:3]) < 2.0 ** 128).all() and held[0] == -held[1] >= 1.5 * 2.0 ** 127
