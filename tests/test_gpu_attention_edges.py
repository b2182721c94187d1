"""Calls of the attention over the NVFP4 cache that its documentation allows and that lie at an edge:
refused slots in every place of the list, extreme positions, caps and queries."""
import math

import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
from gpu_helpers import device_status
from test_gpu_attention import D, assert_close, build, held, queries, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,tokens", [([1, 0], [61, 128]), ([1, 1, 0], [61, 7, 128]), ([1, 0, 1], [59, 128, 1]),
                                          ([2, 0], [200, 128]), ([2, 1, 0], [200, 61, 128])])
@pytest.mark.parametrize("tq,group", [(1, 1), (1, 2), (3, 3), (12, 1), (40, 1), (200, 1)])
def test_refused_slots_before_good_ones(cuda_dev, slots, tokens, tq, group):
    """A slot whose recorded count differs counts as masked wherever it stands in the list: the rest
    gives what it gives alone, but for the grouping of the same sums, so the binary64 bounds hold."""
    cache = build(2, 256, [128, 60, 256], 41)
    q = queries(tq, 2 * group, tq)
    o, lse = torch.full_like(q, 3.0), torch.zeros(2 * group, tq, device="cuda")
    nv.kv_window_attention(cache, slots, tokens, q, 0.1, o, lse_out=lse)
    assert device_status() == nv.ERR_SHAPE
    k, v = held(cache, 0, 128)
    assert_close(o, lse, reference(q, k, v, torch.ones(tq, 128, dtype=torch.bool), 0.1))


@pytest.mark.parametrize("n", [1, 20, 33, 64, 100])
@pytest.mark.parametrize("tq", [12, 130, 300])
@pytest.mark.parametrize("kw", [dict(causal=True), dict(causal=True, window=2 ** 31 - 2), dict(window=5)])
def test_positions_at_both_ends(cuda_dev, n, tq, kw):
    """Queries at position 0 and at the last one, keys at the last positions: no number that the mask
    is made of leaves 32 bits."""
    cache = build(1, 128, [n], 5)
    pos = torch.zeros(tq, dtype=torch.int32, device="cuda")
    pos[::2] = 2 ** 31 - 2
    run(cache, [0], [n], queries(tq, 1, 3), q_pos=pos, slot_pos=[2 ** 31 - 1 - n], **kw)
    run(cache, [0], [n], queries(tq, 1, 4), q_pos=pos, **kw)
