"""Refusals of the layer steps and of attention over the cache at the ends of the arguments' ranges,
before any device work.  CPU only."""
import ctypes

import pytest

import nvfp4_w4a4_quantized_amax_b200 as nv
from test_layer_args import _attend


@pytest.mark.parametrize("tree", [False, True])
def test_first_query_position_near_the_end_of_int64(tree):
    for q_pos in ((1 << 63) - 1, (1 << 63) - 3, 1 << 62, 1 << 32, (1 << 31) - 3):
        assert _attend(tree=tree, q_pos=q_pos) == nv.ERR_SHAPE, q_pos  # of three queries
    for pos in ((1 << 63) - 1, 1 << 32):
        assert _attend(tree=tree, slot_pos_host=(ctypes.c_int64 * 2)(0, pos)) == nv.ERR_SHAPE
