"""Attention over the NVFP4 cache and over drafted tokens, against binary64 softmax attention on
the exact values the cache holds."""
import math

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
from gpu_helpers import device_status

pytestmark = pytest.mark.gpu

D = 128
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def build(heads, chunk, fills, seed, v_scale=None, k_mean=3.0):
    """A cache filled through kv_quant_append; slots hold other garbage (NaN scale bytes among it)
    behind their tokens.  v_scale[s]: factor of the slot's V."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cache = nv.KVCache(heads, D, chunk, len(fills))
    cache.buffer.fill_(0x7F)
    mean = k_mean * torch.randn(heads, D, device="cuda", generator=gen)
    for s, n in enumerate(fills):
        k = torch.randn(n, heads, D, device="cuda", generator=gen) + mean
        v = torch.randn(n, heads, D, device="cuda", generator=gen) * (1.0 if v_scale is None else v_scale[s])
        nv.kv_quant_append(cache, k.bfloat16(), v.bfloat16(), s)
    torch.cuda.synchronize()
    return cache


def held(cache, slot, n):
    """(K^, V^) of a slot's first n tokens in binary64, [n, heads, 128], unrounded."""
    kc, ks, vc, vs, mu, g = cache.slot_views(slot)
    out = []
    for codes, scales, gs in ((kc, ks, g[0]), (vc, vs, g[1])):
        b = codes.view(-1, cache.heads, D // 2)[:n].cpu()
        e = torch.stack([E2M1[(b & 15).long()], E2M1[(b >> 4).long()]], -1).view(n, cache.heads, D // 16, 16)
        s = scales.view(-1, cache.heads, D // 16)[:n].contiguous().view(torch.float8_e4m3fn).cpu().double()
        out.append((e * s[..., None]).view(n, cache.heads, D) * gs.cpu().double())
    return out[0] + mu.cpu().double().view(cache.heads, D), out[1]


def reference(q, k, v, seen, scale, cap=0.0, slopes=None, dist=None):
    """(O, lse, tolerance of O, tolerance of lse), binary64; q [tq, hq, 128], k, v [Tk, h, 128],
    seen and dist [tq, Tk].

    Tolerances: the weights are rounded to binary16: half a step, 2^-11 of their value, and half the
    smallest step, 2^-25, where they are small; a row's largest weight is at least 2^10 there, so
    that is 2^-35 of it.  A score is an FP32 sum on the tensor cores of 128 products plus
    the mean's part; taking 2^-19 of the sum of absolute products (eight accumulations of a
    tensor-core step of 2^-22 each, and the mean's 128 additions of 2^-24 cancel less than that),
    2^-20 of the cap and 2^-22 of the biased score, it moves p by twice that, relatively.  O is
    then rounded to bf16: half a step, 2^-8."""
    tq, hq, _ = q.shape
    group = hq // k.shape[1]
    o, tol = torch.zeros(tq, hq, D, dtype=torch.float64), torch.zeros(tq, hq, D, dtype=torch.float64)
    lse, ltol = torch.zeros(hq, tq, dtype=torch.float64), torch.zeros(hq, tq, dtype=torch.float64)
    for h in range(hq):
        kk, vv, qq = k[:, h // group], v[:, h // group], q[:, h].double().cpu()
        x = qq @ kk.T * scale
        err = 2.0 ** -19 * (qq.abs() @ kk.abs().T + 4 * qq.abs().sum(-1, keepdim=True)) * abs(scale)
        if cap:
            x = cap * torch.tanh(x / cap)
            err = err + 2.0 ** -20 * cap
        if slopes is not None:
            x = x - float(slopes[h]) * dist.abs()
            err = err + 2.0 ** -22 * float(slopes[h]) * dist.abs()
        err = (err + 2.0 ** -22 * x.abs()).masked_fill(~seen, 0.0).amax(-1)
        x = x.masked_fill(~seen, -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), 0.0, top)
        p = torch.exp(x - top)
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
        o[:, h] = p @ vv
        weight = (p * (2.0 ** -11 + 2 * err[:, None])) + seen * 2.0 ** -35
        tol[:, h] = weight @ vv.abs() + 2.0 ** -8 * o[:, h].abs() + 1e-30
        tol[:, h] += 2.0 ** -8 * tol[:, h]
        lse[h] = (top + torch.log(total))[:, 0]
        ltol[h] = err + 2.0 ** -20 * (1 + torch.where(torch.isinf(lse[h]), 0.0, lse[h].abs()))
    return o, lse, tol, ltol


def assert_close(o, lse, ref):
    ro, rl, tol, ltol = ref
    bad = (o.double().cpu() - ro).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} outputs off, first {bad.nonzero()[0].tolist()}"
    if lse is not None:
        got = lse.double().cpu()
        none = torch.isinf(rl)
        assert torch.equal(torch.isinf(got) & (got < 0), none)
        assert bool(((got - rl).abs()[~none] <= ltol[~none]).all())


def queries(tq, heads, seed, pad=0, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = (torch.randn(tq, heads * D + pad, device="cuda", generator=gen) * scale).bfloat16()
    return torch.as_strided(q, (tq, heads, D), (heads * D + pad, D, 1))


def run(cache, slots, tokens, q, scale=D ** -0.5, pad=0, stream=None, **kw):
    tq, hq, _ = q.shape
    out = torch.full((tq + 2, hq * D + pad), 3.0, dtype=torch.bfloat16, device="cuda")  # guarded by rows and columns
    o = torch.as_strided(out, (tq, hq, D), (hq * D + pad, D, 1), hq * D + pad)
    lse = torch.full((hq, tq), 77.0, device="cuda")
    torch.cuda.synchronize()
    nv.kv_window_attention(cache, slots, tokens, q, scale, o, lse_out=lse, stream=stream, **kw)
    torch.cuda.synchronize()
    assert bool((out[0] == 3.0).all()) and bool((out[-1] == 3.0).all()) and bool((out[:, hq * D:] == 3.0).all())
    k, v = (torch.cat(t) for t in zip(*(held(cache, s, n) for s, n in zip(slots, tokens))))
    pos = kw.get("slot_pos")
    if pos is None:
        pos = np.concatenate([[0], np.cumsum(tokens)[:-1]])
    kp = torch.cat([torch.arange(a, a + n) for a, n in zip(pos, tokens)])
    q_pos = kw.get("q_pos", 0)
    qp = q_pos.cpu().long() if isinstance(q_pos, torch.Tensor) else torch.arange(tq) + q_pos
    dist = (qp[:, None] - kp[None]).double()
    seen = torch.ones(tq, len(kp), dtype=torch.bool)
    if kw.get("causal"):
        seen &= dist >= 0
    if kw.get("window"):
        seen &= dist < kw["window"]
    if kw.get("prefix"):
        seen |= (kp < kw["prefix"])[None]
    if kw.get("q_doc") is not None:
        seen &= kw["q_doc"].cpu()[:, None] == kw["k_doc"].cpu()[None]
    ref = reference(q, k, v, seen, scale, kw.get("softcap", 0.0), kw.get("slopes"), dist)
    assert_close(o, lse, ref)
    assert device_status() == nv.OK
    return o, lse, seen


MASKS = {
    "all": dict(),
    "causal": dict(causal=True, q_pos=150),
    "causal, early": dict(causal=True, q_pos=0),
    "sliding": dict(causal=True, window=40, q_pos=200),
    "window of one": dict(causal=True, window=1, q_pos=100),
    "prefix": dict(causal=True, prefix=70, q_pos=20),
    "prefix and window": dict(causal=True, window=30, prefix=5, q_pos=160),
    "cap": dict(softcap=4.0),
    "cap and causal": dict(softcap=20.0, causal=True, q_pos=60),
    "gaps": dict(causal=True, slot_pos=[500, 0, 1000], q_pos=990, window=600),
    "nothing": dict(causal=True, slot_pos=[5000, 6000, 7000], q_pos=0),
}


@pytest.mark.parametrize("mask", list(MASKS))
@pytest.mark.parametrize("tq,group", [(1, 1), (1, 4), (5, 3), (40, 1), (130, 2), (300, 1)])
def test_masks(cuda_dev, mask, tq, group):
    """Three slots out of order with partial fills (201 keys); 1 to 300 rows a cache head."""
    cache = build(2, 128, [13, 128, 60], 3)
    run(cache, [1, 0, 2], [128, 13, 60], queries(tq, 2 * group, tq + group), **MASKS[mask])


@pytest.mark.parametrize("tq,group", [(1, 1), (3, 8), (70, 2)])
def test_bias_and_documents(cuda_dev, tq, group):
    cache = build(3, 100, [100, 37], 5)
    hq = 3 * group
    slopes = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device="cuda") / hq)
    run(cache, [0, 1], [100, 37], queries(tq, hq, 1), slopes=slopes, q_pos=64)
    run(cache, [0, 1], [100, 37], queries(tq, hq, 2), slopes=slopes, q_pos=64, causal=True, softcap=10.0)
    k_doc = (torch.arange(137, device="cuda") // 30).int()
    q_doc = (torch.arange(tq, device="cuda") // 7 - 1).int()  # -1: in no document
    _, lse, seen = run(cache, [0, 1], [100, 37], queries(tq, hq, 3), q_doc=q_doc, k_doc=k_doc)
    assert bool(torch.isinf(lse).any()) == bool((~seen.any(-1)).any())
    run(cache, [0, 1], [100, 37], queries(tq, hq, 4), q_doc=q_doc, k_doc=k_doc, causal=True, q_pos=3, slopes=slopes)


def test_query_positions_in_any_order(cuda_dev):
    cache = build(1, 256, [256, 100], 9)
    pos = torch.tensor([300, 5, 0, 2000, 260, 17, 17], dtype=torch.int32, device="cuda")
    for kw in (dict(causal=True), dict(causal=True, window=64), dict(window=64)):
        run(cache, [0, 1], [256, 100], queries(7, 4, 2), q_pos=pos, **kw)


@pytest.mark.parametrize("fills", [[1], [1, 1, 1], [31, 33, 32], [8] * 40, [64, 1, 127, 128, 3]])
@pytest.mark.parametrize("tq", [1, 17, 129])
def test_short_slots(cuda_dev, fills, tq):
    cache = build(2, 128, fills, len(fills))
    order = list(np.random.default_rng(1).permutation(len(fills)))
    slots, tokens = [int(s) for s in order], [fills[s] for s in order]
    run(cache, slots, tokens, queries(tq, 2, 3, pad=8), pad=24)
    slots, tokens = (slots + slots)[:64], (tokens + tokens)[:64]  # the same index twice
    run(cache, slots, tokens, queries(tq, 4, 4), causal=True, q_pos=2)


@pytest.mark.parametrize("tq,heads,group", [(1, 1, 1), (2, 3, 5), (64, 2, 1), (257, 1, 3), (33, 24, 1)])
def test_split_keys(cuda_dev, tq, heads, group):
    """Windows long enough to be split over CTAs and joined."""
    cache = build(heads, 2048, [2048, 1999, 700], 17)
    run(cache, [0, 1, 2], [2048, 1999, 700], queries(tq, heads * group, 5))
    run(cache, [2, 0], [700, 2048], queries(tq, heads * group, 6), causal=True, q_pos=2000, window=900)


@pytest.mark.parametrize("tq", [1, 200])
def test_value_scales_far_apart(cuda_dev, tq):
    """Slots whose V differ by many orders of magnitude, zeros among them: each row's result is as
    exact as its own values allow, whichever slots it sees."""
    cache = build(2, 64, [64] * 5, 23, v_scale=[1e-8, 1.0, 0.0, 1e6, 1e-3])
    docs = torch.arange(5, device="cuda").repeat_interleave(64).int()
    q_doc = (torch.arange(tq, device="cuda") % 5).int()
    for order in ([0, 1, 2, 3, 4], [3, 2, 1, 4, 0], [2, 0, 4, 1, 3]):
        run(cache, order, [64] * 5, queries(tq, 2, 1))
        k_doc = docs.view(5, 64)[order].flatten()
        run(cache, order, [64] * 5, queries(tq, 2, 2), q_doc=q_doc, k_doc=k_doc)
    zeros = build(1, 64, [64, 20], 29, v_scale=[0.0, 0.0])
    o, _, _ = run(zeros, [0, 1], [64, 20], queries(tq, 1, 3))
    assert bool((o == 0).all())


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -120, 2.0 ** 60, 30.0])
@pytest.mark.parametrize("tq", [2, 140])
def test_query_scales(cuda_dev, scale, tq):
    """Rows of zeros, tiny and huge queries (with a softmax scale to match), very peaked rows."""
    cache = build(1, 128, [128, 50], 31)
    factor = D ** -0.5 / (scale if scale not in (0.0, 30.0) else 1.0)
    run(cache, [0, 1], [128, 50], queries(tq, 2, 8, scale=scale), scale=factor)
    run(cache, [0, 1], [128, 50], queries(tq, 2, 8, scale=scale), scale=-factor)


@pytest.mark.parametrize("tq", [1, 12, 200])
def test_wide_caps(cuda_dev, tq):
    """A cap far above the scores changes them by a share of themselves, not of the cap: 2^30 is
    no cap at all to 2^-40, so the uncapped bounds hold."""
    cache = build(1, 256, [256, 130], 71)
    q = queries(tq, 1, 5)
    o, lse = torch.empty_like(q), torch.empty(1, tq, device="cuda")
    nv.kv_window_attention(cache, [0, 1], [256, 130], q, D ** -0.5, o, lse_out=lse, softcap=2.0 ** 30)
    k, v = (torch.cat(t) for t in zip(held(cache, 0, 256), held(cache, 1, 130)))
    assert_close(o, lse, reference(q, k, v, torch.ones(tq, 386, dtype=torch.bool), D ** -0.5))
    parents = torch.arange(-1, tq - 1, dtype=torch.int32, device="cuda")  # the drafts' own scores
    kn, vn = queries(tq, 1, 6), queries(tq, 1, 7)
    nv.kv_tree_attention(cache, [], [], q, kn, vn, parents, D ** -0.5, o, lse_out=lse, softcap=2.0 ** 30)
    assert_close(o, lse, reference(q, kn.double().cpu(), vn.double().cpu(),
                                   torch.ones(tq, tq, dtype=torch.bool).tril(), D ** -0.5))


@pytest.mark.parametrize("tq", [8, 200])
def test_cap_of_unlike_rows(cuda_dev, tq):
    """Rows far below the cap next to a row at it: their error is a share of their own scores (the
    bound counts 2^-20 of them in place of 2^-20 of the cap)."""
    cache = build(1, 256, [256], 73)
    q = queries(tq, 1, 8)
    q[3] *= 4096
    cap, seen = 8192.0, torch.ones(tq, 256, dtype=torch.bool)
    o, lse = torch.empty_like(q), torch.empty(1, tq, device="cuda")
    nv.kv_window_attention(cache, [0], [256], q, D ** -0.5, o, lse_out=lse, softcap=cap)
    k, v = held(cache, 0, 256)
    x = q.double().cpu()[:, 0] @ k[:, 0].T * D ** -0.5
    small = [i for i in range(tq) if i != 3]
    assert x[3].abs().max() > cap > 100 * x[small].abs().max()
    want = torch.logsumexp(cap * torch.tanh(x / cap), -1)
    err = (2.0 ** -19 * D ** -0.5 * (q.double().cpu()[:, 0].abs() @ k[:, 0].abs().T
                                      + 4 * q.double().cpu()[:, 0].abs().sum(-1, keepdim=True))
           + 2.0 ** -20 * x.abs()).amax(-1) + 2.0 ** -20 * (1 + want.abs())
    assert bool(((lse[0].double().cpu() - want).abs() <= err)[small].all())
    ref = reference(q, k, v, seen, D ** -0.5, cap)
    assert_close(o, lse, ref)


@pytest.mark.parametrize("tq", [3, 150])
def test_nonfinite_queries_stay_in_their_rows(cuda_dev, tq):
    cache = build(2, 128, [128, 128], 37)
    q = queries(tq, 2, 1)
    clean, _, _ = run(cache, [0, 1], [128, 128], q)
    q[1, 0, 5] = math.nan
    q[2, 1, 7] = math.inf
    o = torch.empty_like(q)
    lse = torch.empty(2, tq, device="cuda")
    nv.kv_window_attention(cache, [0, 1], [128, 128], q, D ** -0.5, o, lse_out=lse)
    bad = torch.zeros(tq, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert bool(torch.isnan(o[1, 0]).all()) and bool(torch.isnan(lse[0, 1]))
    assert torch.equal(o[~bad], clean[~bad])
    # a row that sees nothing is empty whatever its query holds
    doc = torch.zeros(tq, dtype=torch.int32, device="cuda")
    doc[1] = 9
    nv.kv_window_attention(cache, [0, 1], [128, 128], q, D ** -0.5, o, lse_out=lse, q_doc=doc,
                           k_doc=torch.zeros(256, dtype=torch.int32, device="cuda"))
    assert bool((o[1] == 0).all()) and bool((lse[:, 1] == -math.inf).all())


@pytest.mark.parametrize("tq", [1, 200])
def test_slot_with_another_count(cuda_dev, tq):
    cache = build(1, 128, [128, 60], 41)
    q = queries(tq, 1, 1)
    o, want = torch.empty_like(q), torch.empty_like(q)
    nv.kv_window_attention(cache, [0], [128], q, 0.1, want)
    nv.kv_window_attention(cache, [0, 1], [128, 61], q, 0.1, o)
    assert device_status() == nv.ERR_SHAPE
    assert torch.equal(o, want)
    nv.kv_window_attention(cache, [1], [61], q, 0.1, o)
    assert device_status() == nv.ERR_SHAPE and bool((o == 0).all())


@pytest.mark.parametrize("tq", [1, 130])
def test_streams_graphs_and_workspaces(cuda_dev, tq):
    cache = build(4, 1024, [1024, 900], 43)
    q = queries(tq, 4, 1)
    run(cache, [0, 1], [1024, 900], q, stream=torch.cuda.Stream())
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(nv.kv_attention_workspace_bytes(cache, [1024, 900], tq, 4), dtype=torch.uint8, device="cuda")
    nv.kv_window_attention(cache, [0, 1], [1024, 900], q, 0.1, o, workspace=ws)  # loads what a capture may not
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_window_attention(cache, [0, 1], [1024, 900], q, 0.1, o, workspace=ws)
        nv.kv_window_attention(cache, [1], [900], q, 0.1, o2)  # its own workspace, from the graph's pool
    for i in range(3):
        q.copy_(queries(tq, 4, 50 + i))
        ws.fill_(0xFF)  # contents mean nothing
        graph.replay()
        want, want2 = torch.empty_like(q), torch.empty_like(q)
        nv.kv_window_attention(cache, [0, 1], [1024, 900], q, 0.1, want)
        nv.kv_window_attention(cache, [1], [900], q, 0.1, want2)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(o2, want2)


def test_many_queries_without_workspace(cuda_dev):
    cache = build(2, 64, [64, 20], 61)
    assert nv.kv_attention_workspace_bytes(cache, [64, 20], 1500, 4) == 0
    run(cache, [0, 1], [64, 20], queries(1500, 4, 1), causal=True)


def test_no_queries(cuda_dev):
    cache = build(1, 64, [64], 1)
    q = torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    nv.kv_window_attention(cache, [0], [64], q, 0.1, torch.empty_like(q))
    new = torch.empty(0, 1, D, dtype=torch.bfloat16, device="cuda")
    nv.kv_tree_attention(cache, [0], [64], q, new, new, torch.empty(0, dtype=torch.int32, device="cuda"), 0.1,
                         torch.empty_like(q))
    assert device_status() == nv.OK


@pytest.mark.parametrize("tq", [1, 256])
def test_agrees_with_scores_and_context(cuda_dev, tq):
    """The one-pass call against the framework's two calls with a softmax between them: those take
    K^ and V^ rounded to bf16 (2^-8 each) and bf16 weights (2^-8)."""
    cache = build(2, 512, [512, 200], 47, k_mean=1.0)
    q = queries(tq, 2, 1, scale=1.0)
    s = torch.empty(2, tq, 712, device="cuda")
    nv.kv_window_scores(cache, [0, 1], [512, 200], q, D ** -0.5, s)
    p = torch.softmax(s, -1).bfloat16()
    two = torch.empty(tq, 2, D, device="cuda")
    nv.kv_window_context(cache, [0, 1], [512, 200], p, two)
    o, _, _ = run(cache, [0, 1], [512, 200], q)
    k, v = (torch.cat(t) for t in zip(*(held(cache, i, n) for i, n in ((0, 512), (1, 200)))))
    spread = 2.0 ** -8 * (q.double().cpu().abs().transpose(0, 1) @ k.abs().permute(1, 2, 0)).amax(-1) * D ** -0.5
    bound = (2 * spread + 4 * 2.0 ** -8)[..., None] * torch.einsum("htk,khd->htd", p.double().cpu(), v.abs())
    assert bool(((o.double() - two.double()).abs().cpu() <= bound.transpose(0, 1)).all())


# ------------------------------------------------------------------------ drafted tokens


def run_tree(cache, slots, tokens, parents, hq, seed, scale=D ** -0.5, poison=False, pad=0, q_pos=None, **kw):
    n, h = len(parents), cache.heads
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = queries(n, hq, seed, pad=pad)
    k_new = (torch.randn(n, h, D, device="cuda", generator=gen) * 2).bfloat16()
    v_new = torch.randn(n, h, D, device="cuda", generator=gen).bfloat16()
    depth, seen = [], np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        if p >= 0:
            seen[i] = seen[p]
        seen[i, i] = True
    start = sum(tokens) if q_pos is None else q_pos
    o = torch.full_like(q, 3.0)
    lse = torch.zeros(hq, n, device="cuda")
    par = torch.tensor(parents, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    nv.kv_tree_attention(cache, slots, tokens, q, k_new, v_new, par, scale, o, lse_out=lse, q_pos=start, **kw)
    torch.cuda.synchronize()
    pos = kw.get("slot_pos")
    if pos is None:
        pos = np.concatenate([[0], np.cumsum(tokens)[:-1]]).astype(int)
    parts = [held(cache, s, t) for s, t in zip(slots, tokens)]
    k = torch.cat([a for a, _ in parts] + [k_new.double().cpu()])
    v = torch.cat([b for _, b in parts] + [v_new.double().cpu()])
    qp = torch.tensor(depth, dtype=torch.long) + start
    kp = torch.cat([torch.arange(a, a + t) for a, t in zip(pos, tokens)] + [qp])
    dist = (qp[:, None] - kp[None]).double()
    see = torch.cat([torch.ones(n, sum(tokens), dtype=torch.bool), torch.from_numpy(seen)], 1)
    if kw.get("window"):
        see &= dist < kw["window"]
    ref = reference(q, k, v, see, scale, kw.get("softcap", 0.0), kw.get("slopes"), dist)
    assert_close(o, lse, ref)
    assert device_status() == nv.OK
    if poison:  # what a row does not see cannot reach it
        k_new[-1], v_new[-1] = math.nan, math.inf
        o2 = torch.full_like(q, 3.0)
        nv.kv_tree_attention(cache, slots, tokens, q, k_new, v_new, par, scale, o2, q_pos=start, **kw)
        assert torch.equal(o2[:-1], o[:-1]) and bool(torch.isnan(o2[-1]).all())


TREES = {
    "one": [-1],
    "chain": list(range(-1, 22)),
    "long chain": list(range(-1, 299)),
    "roots": [-1] * 9,
    "binary": [-1, -1] + [(i - 2) // 2 for i in range(2, 63)],
    "random": [-1] + [int(p) for p in np.random.default_rng(0).integers(-1, np.arange(1, 130))],
}


@pytest.mark.parametrize("tree", list(TREES))
@pytest.mark.parametrize("group", [1, 4])
def test_tree(cuda_dev, tree, group):
    cache = build(2, 200, [200, 45], 51)
    run_tree(cache, [0, 1], [200, 45], TREES[tree], 2 * group, 1, poison=len(TREES[tree]) > 1)
    run_tree(cache, [1], [45], TREES[tree], 2 * group, 2, softcap=15.0, pad=8)
    run_tree(cache, [], [], TREES[tree], 2 * group, 3)  # no window yet


def test_tree_bias_window_and_positions(cuda_dev):
    cache = build(1, 128, [128, 100], 53)
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.02], device="cuda")
    for tree in ("chain", "random"):
        run_tree(cache, [0, 1], [128, 100], TREES[tree], 4, 1, slopes=slopes)
        run_tree(cache, [0, 1], [128, 100], TREES[tree], 4, 2, window=9)
        run_tree(cache, [0, 1], [128, 100], TREES[tree], 4, 3, window=50, slopes=slopes, slot_pos=[0, 1000], q_pos=1100)


def test_tree_long_window(cuda_dev):
    cache = build(3, 4096, [4096, 3000], 57)
    run_tree(cache, [0, 1], [4096, 3000], TREES["binary"], 3, 1)
    run_tree(cache, [0, 1], [4096, 3000], [-1], 12, 2)


def test_tree_wrong_parents(cuda_dev):
    """A parent that does not come before its child counts as none and is reported."""
    cache = build(1, 64, [64], 59)
    q = queries(4, 1, 1)
    new = torch.randn(4, 1, D, device="cuda").bfloat16()
    out = []
    for parents in ([-1, 1, 7, -9], [-1, -1, -1, -1]):
        o = torch.empty_like(q)
        nv.kv_tree_attention(cache, [0], [64], q, new, new, torch.tensor(parents, dtype=torch.int32, device="cuda"),
                             0.1, o, q_pos=64, window=100)
        out.append(o)
        assert device_status() == (nv.ERR_SHAPE if parents[1] == 1 else nv.OK)
    assert torch.equal(out[0], out[1])


def test_tree_equals_causal_window(cuda_dev):
    """A chain of drafts gives what the window call gives once the same tokens are in the cache, up
    to the cache's 4 bits: compared on tokens that 4 bits hold exactly (a mean of 0, codes times
    one scale)."""
    n = 32
    table = E2M1[[1, 2, 4, 5, 6, 7]].float()
    gen = torch.Generator().manual_seed(3)
    half = table[torch.randint(0, 6, (n // 2, 1, D), generator=gen)]
    half[:, :, ::16] = 6.0  # every block's largest is 6, so every block scale is the same
    k = torch.cat([half, -half]).cuda().bfloat16()  # mean 0
    v = torch.cat([half.flip(0), half]).cuda().bfloat16()
    cache = nv.KVCache(1, D, n, 1)
    nv.kv_quant_append(cache, k, v, 0)
    hk, hv = held(cache, 0, n)
    assert torch.allclose(hk, k.double().cpu(), rtol=1e-6) and torch.allclose(hv, v.double().cpu(), rtol=1e-6)
    q = queries(n, 2, 5)
    a, b = torch.empty_like(q), torch.empty_like(q)
    nv.kv_window_attention(cache, [0], [n], q, 0.05, a, causal=True)
    nv.kv_tree_attention(cache, [], [], q, k, v, torch.arange(-1, n - 1, dtype=torch.int32, device="cuda"), 0.05, b)
    ref = reference(q, hk, hv, torch.tril(torch.ones(n, n, dtype=torch.bool)), 0.05)
    assert_close(a, None, ref)
    assert_close(b, None, ref)
