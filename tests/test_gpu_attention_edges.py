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


@pytest.mark.parametrize("cap", [2.0 ** 60, 2.0 ** 110, 2.0 ** 120, 2.0 ** 127, 3.4e38])
@pytest.mark.parametrize("tq", [1, 12, 200])
def test_caps_beyond_every_score(cuda_dev, cap, tq):
    """tanh changes a score of at most 2^9 by less than 2^-100 of it under these caps: the uncapped
    bounds hold, for keys of the window and for drafts."""
    cache = build(1, 256, [256, 130], 71)
    q = queries(tq, 1, 5)
    o, lse = torch.empty_like(q), torch.empty(1, tq, device="cuda")
    nv.kv_window_attention(cache, [0, 1], [256, 130], q, D ** -0.5, o, lse_out=lse, softcap=cap)
    k, v = (torch.cat(t) for t in zip(held(cache, 0, 256), held(cache, 1, 130)))
    assert_close(o, lse, reference(q, k, v, torch.ones(tq, 386, dtype=torch.bool), D ** -0.5))
    parents = torch.arange(-1, tq - 1, dtype=torch.int32, device="cuda")
    kn, vn = queries(tq, 1, 6), queries(tq, 1, 7)
    nv.kv_tree_attention(cache, [], [], q, kn, vn, parents, D ** -0.5, o, lse_out=lse, softcap=cap)
    assert_close(o, lse, reference(q, kn.double().cpu(), vn.double().cpu(),
                                   torch.ones(tq, tq, dtype=torch.bool).tril(), D ** -0.5))
    assert device_status() == nv.OK


@pytest.mark.parametrize("cap", [2.0 ** -30, 2.0 ** -64, 2.0 ** -126, 1e-42])
@pytest.mark.parametrize("size", [1.5, 2.0 ** 20])
@pytest.mark.parametrize("tq", [1, 12, 200])
def test_caps_below_every_score(cuda_dev, cap, size, tq):
    """Scores within 2^-30 of 0: all weights are one to 2^-29, each rounded to binary16 by at most
    2^-11, and O to bf16 by 2^-8; lse is the logarithm of the number of keys in FP32."""
    cache = build(1, 256, [256, 130], 72)
    q = queries(tq, 1, 5, scale=size)
    o, lse = torch.empty_like(q), torch.empty(1, tq, device="cuda")

    def check(v, seen):
        p = seen.double() / seen.sum(-1, keepdim=True)
        want, tol = p @ v[:, 0], p @ v[:, 0].abs() * 2.0 ** -10
        assert bool(((o[:, 0].double().cpu() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
        n = seen.sum(-1).double().log()
        assert bool(((lse[0].double().cpu() - n).abs() <= 2.0 ** -20 * (1 + n)).all())

    nv.kv_window_attention(cache, [0, 1], [256, 130], q, D ** -0.5, o, lse_out=lse, softcap=cap)
    check(torch.cat([held(cache, 0, 256)[1], held(cache, 1, 130)[1]]), torch.ones(tq, 386, dtype=torch.bool))
    parents = torch.arange(-1, tq - 1, dtype=torch.int32, device="cuda")
    kn, vn = queries(tq, 1, 6), queries(tq, 1, 7)
    nv.kv_tree_attention(cache, [], [], q, kn, vn, parents, D ** -0.5, o, lse_out=lse, softcap=cap)
    check(vn.double().cpu(), torch.ones(tq, tq, dtype=torch.bool).tril())
    assert device_status() == nv.OK


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("tq", [2, 12, 100, 200])
def test_nonfinite_queries_are_nan(cuda_dev, tq, softcap, value):
    """A query with a NaN or Inf gives NaN where it sees a key, also where all its scores would be
    -Inf (one visible key) or finite (a cap); it is empty where it sees none; other rows stay."""
    cache = build(2, 128, [128], 37)
    q = queries(tq, 2, 1)
    clean, odd = q.clone(), torch.zeros(tq, dtype=torch.bool, device="cuda")
    odd[::2] = True
    q[odd, :, 77] = value
    o, lse, want = torch.empty_like(q), torch.empty(2, tq, device="cuda"), torch.empty_like(q)
    for key in range(0, 128, 9):  # the only one that is seen
        pos = torch.full((tq,), key, dtype=torch.int32, device="cuda")
        kw = dict(causal=True, window=1, softcap=softcap, q_pos=pos)
        nv.kv_window_attention(cache, [0], [128], clean, D ** -0.5, want, **kw)
        nv.kv_window_attention(cache, [0], [128], q, D ** -0.5, o, lse_out=lse, **kw)
        assert bool(torch.isnan(o[odd]).all()) and bool(torch.isnan(lse[:, odd]).all())
        assert torch.equal(o[~odd], want[~odd]) and bool(torch.isfinite(lse[:, ~odd]).all())
    nv.kv_window_attention(cache, [0], [128], q, D ** -0.5, o, lse_out=lse, causal=True, slot_pos=[5000],
                           softcap=softcap)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    parents = torch.full((tq,), -1, dtype=torch.int32, device="cuda")
    kn, vn = queries(tq, 2, 6), queries(tq, 2, 7)
    for slots, tokens in (([], []), ([0], [128])):
        nv.kv_tree_attention(cache, slots, tokens, clean, kn, vn, parents, D ** -0.5, want, softcap=softcap)
        nv.kv_tree_attention(cache, slots, tokens, q, kn, vn, parents, D ** -0.5, o, lse_out=lse, softcap=softcap)
        assert bool(torch.isnan(o[odd]).all()) and bool(torch.isnan(lse[:, odd]).all())
        assert torch.equal(o[~odd], want[~odd]) and bool(torch.isfinite(lse[:, ~odd]).all())
    assert device_status() == nv.OK


@pytest.mark.parametrize("power", [-80, -105, -117])
@pytest.mark.parametrize("tq,group", [(1, 1), (5, 2), (100, 1), (300, 1)])
@pytest.mark.parametrize("scale", [D ** -0.5, 2.0 ** -12])
def test_small_values(cuda_dev, power, tq, group, scale):
    """Values whose g_V is close to FP32's smallest numbers keep their digits, with few and with all of
    the keys counting: in units of 2^power the bounds are the usual ones and bf16's smallest half step,
    2^-134."""
    cache = build(2, 1024, [1024, 500], 75, v_scale=[2.0 ** power] * 2)
    q = queries(tq, 2 * group, 1)
    o, lse = torch.empty_like(q), torch.empty(2 * group, tq, device="cuda")
    nv.kv_window_attention(cache, [0, 1], [1024, 500], q, scale, o, lse_out=lse)
    k, v = (torch.cat(t) for t in zip(held(cache, 0, 1024), held(cache, 1, 500)))
    ro, rl, tol, ltol = reference(q, k, v * 2.0 ** -power, torch.ones(tq, 1524, dtype=torch.bool), scale)
    assert_close(o.double() * 2.0 ** -power, lse, (ro, rl, tol + 2.0 ** (-134 - power), ltol))
