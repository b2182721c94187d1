"""Refusals of the layer steps and of attention over the cache at the ends of the arguments' ranges,
before any device work.  CPU only."""
import ctypes

import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
from test_layer_args import _attend, _cache


@pytest.mark.parametrize("tree", [False, True])
def test_first_query_position_near_the_end_of_int64(tree):
    for q_pos in ((1 << 63) - 1, (1 << 63) - 3, 1 << 62, 1 << 32, (1 << 31) - 3):
        assert _attend(tree=tree, q_pos=q_pos) == nv.ERR_SHAPE, q_pos  # of three queries
    for pos in ((1 << 63) - 1, 1 << 32):
        assert _attend(tree=tree, slot_pos_host=(ctypes.c_int64 * 2)(0, pos)) == nv.ERR_SHAPE


def test_drafts_without_parents():
    cache = nv.KVCache.__new__(nv.KVCache)
    cache.handle, cache.heads, cache.head_dim, cache.buffer = _cache(), 2, 128, torch.zeros(1)
    q, new = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="parents"):
        nv.kv_tree_attention(cache, [0], [64], q, new, new, None, 0.1, torch.zeros_like(q))


def test_first_rope_position_beyond_binary64():
    P, y = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 20)
    for pos0 in ((1 << 63) - 1, (1 << 53) - 3, -(1 << 53) - 1, -(1 << 63)):  # of four tokens
        assert nv.library().nvfp4_rope(P, nv.BF16, 4, 2, 64, 128, P, 64, nv.ROPE_HALF, 1.0, None, pos0, y, 128,
                                       None) == nv.ERR_SHAPE, pos0


def test_positions_that_no_c_integer_holds():
    """Their low 64 bits would be taken for another position."""
    x, table = torch.zeros(4, 2, 32, dtype=torch.bfloat16), nv.RopeTable(16, device="cpu")
    cache = nv.KVCache.__new__(nv.KVCache)
    cache.handle, cache.heads, cache.head_dim, cache.buffer = _cache(), 2, 128, torch.zeros(1)
    q, new = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    parents = torch.full((3,), -1, dtype=torch.int32)
    for pos in (2 ** 64, 2 ** 63, -2 ** 63 - 1):
        with pytest.raises(ValueError, match="position"):
            nv.nvfp4_rope(x, table, pos)
        with pytest.raises(ValueError, match="position"):
            nv.kv_window_attention(cache, [0], [64], q, 0.1, torch.zeros_like(q), q_pos=pos)
        with pytest.raises(ValueError, match="position"):
            nv.kv_tree_attention(cache, [0], [64], q, new, new, parents, 0.1, torch.zeros_like(q), q_pos=pos)
