"""Attention over the NVFP4 cache at the ends of its sizes: windows so long that a split is forced,
many query heads on one cache head; and capped scores held to their own size."""
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
from gpu_helpers import device_status
from test_gpu_attention import D, assert_close, build, held, queries, reference, run, run_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tq,group", [(1, 1), (3, 5), (70, 1), (140, 1)])
def test_windows_beyond_one_list(cuda_dev, tq, group):
    """More keys than one CTA of the many-row form lists (131072), over the last slots of a cache."""
    fills = [65536, 40000, 65536, 301]
    cache = build(1, 65536, fills, 3)
    run(cache, [2, 0, 3, 1], [65536, 65536, 301, 40000], queries(tq, group, 1), causal=True, window=150000,
        q_pos=171000)


def test_sixty_four_full_slots(cuda_dev):
    fills = [2500] * 64
    cache = build(1, 2500, fills, 4)
    run(cache, list(range(63, -1, -1)), fills, queries(2, 2, 1), prefix=2600, window=3000, causal=True, q_pos=159998)
    run(cache, list(range(64)), fills, queries(130, 1, 2), causal=True, q_pos=159870)


@pytest.mark.parametrize("group", [9, 16, 17, 24, 64, 65, 100, 128, 129, 300])
@pytest.mark.parametrize("tq", [1, 2])
def test_many_heads_on_one(cuda_dev, group, tq):
    cache = build(2, 512, [512, 300], 6)
    run(cache, [0, 1], [512, 300], queries(tq, 2 * group, 1), causal=True, q_pos=700, window=600, softcap=20.0)
    run_tree(cache, [0, 1], [512, 300], [-1, 0][:tq], 2 * group, 2)


@pytest.mark.parametrize("tq,group", [(1, 1), (5, 3), (40, 1), (130, 2), (300, 1)])
@pytest.mark.parametrize("cap", [2.0, 30.0, 1e4])
def test_caps_as_shares_of_the_scores(cuda_dev, tq, group, cap):
    """The bounds of the uncapped scores and 2^-20 of each row's largest capped one: tanh is good to
    2^-21 of itself, and its argument's error does not grow (its slope is at most 1)."""
    cache = build(2, 512, [512, 201], 8)
    q = queries(tq, 2 * group, tq)
    o, lse = torch.empty_like(q), torch.empty(2 * group, tq, device="cuda")
    nv.kv_window_attention(cache, [1, 0], [201, 512], q, D ** -0.5, o, lse_out=lse, softcap=cap)
    assert device_status() == nv.OK
    k, v = (torch.cat(t) for t in zip(held(cache, 1, 201), held(cache, 0, 512)))
    seen = torch.ones(tq, 713, dtype=torch.bool)
    ro, rl, _, _ = reference(q, k, v, seen, D ** -0.5, cap)
    qq, scale = q.double().cpu(), D ** -0.5
    for h in range(2 * group):
        kk, vv, qh = k[:, h // group], v[:, h // group], qq[:, h]
        x = cap * torch.tanh(qh @ kk.T * scale / cap)
        err = (2.0 ** -19 * (qh.abs() @ kk.abs().T + 4 * qh.abs().sum(-1, keepdim=True)) * scale).amax(-1)
        err = err + (2.0 ** -20 + 2.0 ** -22) * x.abs().amax(-1)
        p = torch.softmax(x, -1)
        tol = (p * (2.0 ** -11 + 2 * err[:, None]) + 2.0 ** -35) @ vv.abs()
        tol = (tol + 2.0 ** -8 * ro[:, h].abs()) * (1 + 2.0 ** -8)
        assert bool(((o[:, h].double().cpu() - ro[:, h]).abs() <= tol).all())
        assert bool(((lse[h].double().cpu() - rl[h]).abs() <= err + 2.0 ** -20 * (1 + rl[h].abs())).all())


@pytest.mark.parametrize("tq", [1, 12, 140])
def test_cache_beyond_32_bits(cuda_dev, tq):
    """Slots whose codes lie more than 2^32 bytes into the cache."""
    heads, chunk, slots = 32, 65536, 40
    cache = nv.KVCache(heads, D, chunk, slots)
    for s, n in ((39, 100), (1, 60)):
        k, v = (torch.randn(n, heads, D, device="cuda").bfloat16() for _ in range(2))
        nv.kv_quant_append(cache, k, v, s)
    assert 39 * chunk * heads * D // 2 > 1 << 32
    run(cache, [39, 1], [100, 60], queries(tq, heads, 1), causal=True, q_pos=90)
    run_tree(cache, [1, 39], [60, 100], [-1] * min(tq, 20), heads, 2)


@pytest.mark.parametrize("tq", [1, 40, 300])
def test_two_streams_at_once(cuda_dev, tq):
    """Calls that run beside one another, each with its own workspace."""
    cache = build(4, 2048, [2048, 1500], 9)
    qs = [queries(tq, 8, i) for i in range(8)]
    want = [torch.empty_like(q) for q in qs]
    for q, o in zip(qs, want):
        nv.kv_window_attention(cache, [0, 1], [2048, 1500], q, D ** -0.5, o)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], [torch.full_like(q, 3.0) for q in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (q, o) in enumerate(zip(qs, got)):
            nv.kv_window_attention(cache, [0, 1], [2048, 1500], q, D ** -0.5, o, stream=streams[i % 4])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and device_status() == nv.OK
