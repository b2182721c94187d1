"""Host-side rules of the layer steps and of attention over the cache: refusals before any
device work, the rotation frequencies, the binding's own checks.  CPU only."""
import ctypes
import math

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv

P = ctypes.c_void_p(4096)


def _tensor(rows=16, cols=64):
    return nv.nvfp4_tensor(4096, 4096, 4096, rows, cols, ((cols // 2 + 15) // 16) * 16, 0, nv.SF_MMA, 0)


def _norm(x=P, xt=nv.BF16, rows=16, cols=64, ldx=64, res=None, ldr=0, w=P, wt=nv.BF16, eps=1e-6, h=None, ldh=0, g=P,
          out=None, amax=None):
    out = out or _tensor()
    return nv.library().nvfp4_rmsnorm_quantize(x, xt, rows, cols, ldx, res, ldr, w, wt, eps, h, ldh, g,
                                               ctypes.byref(out), amax, None)


def test_rmsnorm_refusals():
    A = ctypes.c_void_p(4098)
    assert _norm(x=None) == nv.ERR_INVALID_ARG
    assert _norm(xt=7) == nv.ERR_INVALID_ARG
    assert _norm(wt=7) == nv.ERR_INVALID_ARG
    for eps in (-1.0, math.nan, math.inf):
        assert _norm(eps=eps) == nv.ERR_INVALID_ARG
    assert _norm(g=None) == nv.ERR_INVALID_ARG  # no scale and nowhere to put max|y|
    assert _norm(rows=17) == nv.ERR_SHAPE
    assert _norm(ldx=48) == nv.ERR_SHAPE
    assert _norm(res=P, ldr=48) == nv.ERR_SHAPE
    assert _norm(h=ctypes.c_void_p(8192), ldh=48) == nv.ERR_SHAPE
    assert _norm(x=A) == nv.ERR_ALIGNMENT
    assert _norm(w=A) == nv.ERR_ALIGNMENT
    assert _norm(ldx=68) == nv.ERR_ALIGNMENT
    assert _norm(res=P, ldr=66) == nv.ERR_ALIGNMENT
    assert _norm(amax=P) == nv.ERR_INVALID_ARG  # max|y| over a scale that is still read
    assert _norm(g=ctypes.c_void_p(8192), amax=ctypes.c_void_p(8192)) == nv.ERR_INVALID_ARG
    # in place with another pitch: rows would overwrite one another
    assert _norm(h=P, ldh=72) == nv.ERR_INVALID_ARG
    bad = _tensor(cols=64)
    bad.cols = 40
    assert _norm(cols=40, out=bad) == nv.ERR_SHAPE


def _freq(rot=64, base=1e4, scaling=nv.ROPE_PLAIN, factor=1.0, original=0, fast=32.0, slow=1.0):
    f, m = (ctypes.c_double * max(1, rot // 2))(), ctypes.c_float()
    st = nv.library().nvfp4_rope_frequencies(rot, base, scaling, factor, original, fast, slow, f, ctypes.byref(m))
    return st, np.array(f), m.value


def test_rope_frequencies():
    for rot in (2, 64, 72, 128):
        i = np.arange(rot // 2)
        f = 1e4 ** (-2.0 * i / rot)
        st, got, m = _freq(rot)
        assert st == nv.OK and m == 1.0 and np.allclose(got, f, rtol=1e-14, atol=0)
        st, got, m = _freq(rot, scaling=nv.ROPE_LINEAR, factor=4.0)
        assert st == nv.OK and m == 1.0 and np.allclose(got, f / 4, rtol=1e-14, atol=0)
    # by parts: fast pairs untouched, slow pairs stretched, monotonic in between
    st, got, m = _freq(128, 5e5, nv.ROPE_BY_PARTS, 8.0, 8192)
    f = 5e5 ** (-2.0 * np.arange(64) / 128)
    turns = 8192 * f / (2 * math.pi)
    assert st == nv.OK and m == np.float32(0.1 * math.log(8.0) + 1.0)
    ratio = got / f
    assert np.allclose(ratio[turns > 40], 1.0, rtol=1e-14) and np.allclose(ratio[turns < 0.8], 1 / 8, rtol=1e-14)
    assert np.all(np.diff(ratio) <= 1e-15)
    lo = math.floor(128 * math.log(8192 / (32 * 2 * math.pi)) / (2 * math.log(5e5)))
    hi = math.ceil(128 * math.log(8192 / (2 * math.pi)) / (2 * math.log(5e5)))
    mid = (lo + hi) // 2
    share = (mid - lo) / (hi - lo)
    assert math.isclose(ratio[mid], share / 8 + 1 - share, rel_tol=1e-12)


def test_rope_frequency_refusals():
    assert _freq(rot=3)[0] == nv.ERR_SHAPE and _freq(rot=0)[0] == nv.ERR_SHAPE
    assert _freq(base=1.0)[0] == nv.ERR_INVALID_ARG and _freq(base=math.inf)[0] == nv.ERR_INVALID_ARG
    assert _freq(scaling=9)[0] == nv.ERR_INVALID_ARG
    assert _freq(scaling=nv.ROPE_LINEAR, factor=0.5)[0] == nv.ERR_INVALID_ARG
    assert _freq(scaling=nv.ROPE_BY_PARTS, factor=4.0, original=0)[0] == nv.ERR_INVALID_ARG
    assert _freq(scaling=nv.ROPE_BY_PARTS, factor=4.0, original=8, fast=1.0, slow=2.0)[0] == nv.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        nv.RopeTable(64, scaling="cubic")
    with pytest.raises(ValueError):
        nv.RopeTable(7)


def _rope(x=P, xt=nv.BF16, tokens=4, heads=2, dim=64, ldx=128, freq=P, rot=64, layout=nv.ROPE_HALF, m=1.0, pos=None,
          y=ctypes.c_void_p(1 << 20), ldy=128):
    return nv.library().nvfp4_rope(x, xt, tokens, heads, dim, ldx, freq, rot, layout, m, pos, 0, y, ldy, None)


def test_rope_refusals():
    assert _rope(x=None) == nv.ERR_INVALID_ARG and _rope(y=None) == nv.ERR_INVALID_ARG
    assert _rope(freq=None) == nv.ERR_INVALID_ARG
    assert _rope(xt=5) == nv.ERR_INVALID_ARG and _rope(layout=2) == nv.ERR_INVALID_ARG
    assert _rope(m=math.nan) == nv.ERR_INVALID_ARG
    assert _rope(rot=66) == nv.ERR_SHAPE and _rope(rot=63) == nv.ERR_SHAPE and _rope(rot=0) == nv.ERR_SHAPE
    assert _rope(tokens=-1) == nv.ERR_SHAPE and _rope(dim=8192, rot=2) == nv.ERR_SHAPE
    assert _rope(heads=1 << 16, ldx=1 << 22, ldy=1 << 22) == nv.ERR_SHAPE
    assert _rope(ldx=127) == nv.ERR_SHAPE and _rope(ldy=64) == nv.ERR_SHAPE
    assert _rope(x=ctypes.c_void_p(4097)) == nv.ERR_ALIGNMENT
    assert _rope(freq=ctypes.c_void_p(4100)) == nv.ERR_ALIGNMENT
    assert _rope(y=P, ldy=160) == nv.ERR_INVALID_ARG  # in place with another pitch


def _cache(heads=2, dim=128, chunk=64, slots=4):
    h = nv.nvfp4_kv_cache()
    st = nv.library().nvfp4_kv_cache_init(ctypes.c_void_p(4096), 1 << 30, heads, dim, chunk, slots, ctypes.byref(h))
    assert st == nv.OK
    return h


def _attend(cache=None, slots=(0, 1), tokens=(64, 5), q=P, tq=3, q_heads=4, ldq=512, o=P, ldo=512, lse=None, n=None,
            tree=False, k_new=P, ld_new=256, parents=P, **at):
    cache = cache or _cache()
    a = nv.nvfp4_attention()
    a.scale = 0.1
    a.workspace, a.workspace_bytes = 4096, 1 << 30
    for k, v in at.items():
        setattr(a, k, v)
    s, t = (ctypes.c_int32 * len(slots))(*slots), (ctypes.c_int32 * len(tokens))(*tokens)
    n = len(slots) if n is None else n
    if tree:
        return nv.library().kv_tree_attention(ctypes.byref(cache), s, t, n, q, tq, q_heads, ldq, k_new, P, ld_new,
                                              parents, ctypes.byref(a), o, ldo, lse, None)
    return nv.library().kv_window_attention(ctypes.byref(cache), s, t, n, q, tq, q_heads, ldq, ctypes.byref(a), o, ldo,
                                            lse, None)


@pytest.mark.parametrize("tree", [False, True])
def test_attention_refusals(tree):
    def f(**kw):
        return _attend(tree=tree, **kw)

    assert f(q=None) == nv.ERR_INVALID_ARG and f(o=None) == nv.ERR_INVALID_ARG
    assert f(slots=(0, 4)) == nv.ERR_INVALID_ARG and f(slots=(0, -1)) == nv.ERR_INVALID_ARG
    assert f(tokens=(64, 65)) == nv.ERR_SHAPE and f(tokens=(0, 1)) == nv.ERR_SHAPE
    assert f(n=65) == nv.ERR_INVALID_ARG and f(n=-1) == nv.ERR_INVALID_ARG
    assert f(q_heads=3) == nv.ERR_SHAPE and f(q_heads=1) == nv.ERR_SHAPE and f(q_heads=0) == nv.ERR_SHAPE
    assert f(tq=-1) == nv.ERR_SHAPE
    assert f(ldq=504) == nv.ERR_SHAPE and f(ldo=504) == nv.ERR_SHAPE
    assert f(ldq=516) == nv.ERR_ALIGNMENT and f(q=ctypes.c_void_p(4104)) == nv.ERR_ALIGNMENT
    assert f(lse=ctypes.c_void_p(4098)) == nv.ERR_ALIGNMENT
    assert f(cache=_cache(dim=64)) == nv.ERR_SHAPE
    assert f(scale=math.nan) == nv.ERR_INVALID_ARG and f(scale=math.inf) == nv.ERR_INVALID_ARG
    assert f(softcap=-1.0) == nv.ERR_INVALID_ARG and f(softcap=math.inf) == nv.ERR_INVALID_ARG
    assert f(reserved=1) == nv.ERR_INVALID_ARG
    assert f(window=-1) == nv.ERR_SHAPE and f(q_pos=-1) == nv.ERR_SHAPE and f(q_pos=(1 << 31) - 2) == nv.ERR_SHAPE
    for pos in ((0, -1), (0, (1 << 31) - 5)):
        assert f(slot_pos_host=(ctypes.c_int64 * 2)(*pos)) == nv.ERR_SHAPE
    assert f(workspace=None) == nv.ERR_INVALID_ARG and f(workspace_bytes=16) == nv.ERR_INVALID_ARG
    assert f(workspace=4100) == nv.ERR_ALIGNMENT
    huge = nv.nvfp4_kv_cache()
    assert nv.library().nvfp4_kv_cache_init(ctypes.c_void_p(4096), 1 << 41, 1, 128, 1 << 20, 1 << 12,
                                            ctypes.byref(huge)) == nv.OK
    assert f(cache=huge, q_heads=2) == nv.ERR_SHAPE  # 2^32 tokens


def test_window_attention_refusals():
    assert _attend(slots=(), tokens=()) == nv.ERR_INVALID_ARG
    assert _attend(causal=2) == nv.ERR_INVALID_ARG
    assert _attend(prefix=-1) == nv.ERR_SHAPE
    assert _attend(q_doc=4096) == nv.ERR_INVALID_ARG and _attend(k_doc=4096) == nv.ERR_INVALID_ARG
    assert _attend(q_doc=4096, k_doc=4098) == nv.ERR_ALIGNMENT
    assert _attend(tq=1 << 30) == nv.ERR_SHAPE


def test_tree_attention_refusals():
    assert _attend(tree=True, parents=None) == nv.ERR_INVALID_ARG
    assert _attend(tree=True, k_new=None) == nv.ERR_INVALID_ARG
    assert _attend(tree=True, tq=1025) == nv.ERR_SHAPE
    assert _attend(tree=True, ld_new=248) == nv.ERR_SHAPE
    assert _attend(tree=True, ld_new=260) == nv.ERR_ALIGNMENT
    for bad in ({"causal": 1}, {"prefix": 1}, {"q_pos_dev": 4096}, {"q_doc": 4096, "k_doc": 4096}):
        assert _attend(tree=True, **bad) == nv.ERR_INVALID_ARG


def test_workspace_sizes():
    cache = nv.KVCache.__new__(nv.KVCache)
    cache.handle = _cache()
    need = nv.kv_attention_workspace_bytes(cache, [64, 5], 3, 4)
    assert need >= 2 * 6 * 129 * 4 and need % 4 == 0
    assert nv.kv_attention_workspace_bytes(cache, [], 1, 2) > 0  # a tree without a window
    assert nv.kv_attention_workspace_bytes(cache, [64], 0, 2) == 0
    assert nv.kv_attention_workspace_bytes(cache, [64], 1024, 2) > 0
    assert nv.kv_attention_workspace_bytes(cache, [64], 1 << 20, 2) == 0  # nothing to join
    for tokens, tq, heads in (([65], 1, 2), ([1], -1, 2), ([1], 1, 3)):
        with pytest.raises(nv.Nvfp4Error):
            nv.kv_attention_workspace_bytes(cache, tokens, tq, heads)


def test_binding_refuses_what_the_calls_cannot_express():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = nv.NVFP4Tensor(4, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_rmsnorm_quantize(x, q, amax_out=torch.zeros(1))
    with pytest.raises(ValueError, match="residual"):
        nv.nvfp4_rmsnorm_quantize(x, q, residual=x.float())
    with pytest.raises(ValueError, match="weight"):
        nv.nvfp4_rmsnorm_quantize(x, q, weight=torch.zeros(32))
    with pytest.raises(ValueError, match="gscale_in"):
        nv.nvfp4_rmsnorm_quantize(x, q, gscale_in=torch.zeros(1, dtype=torch.float64))
    table = nv.RopeTable(16, device="cpu")
    assert table.freq.dtype == torch.float64 and table.freq.shape == (8,)
    t = torch.zeros(4, 2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nv.nvfp4_rope(t, table)
    with pytest.raises(ValueError, match="contiguous heads"):
        nv.nvfp4_rope(t.transpose(1, 2), table)
    with pytest.raises(ValueError, match="positions"):
        nv.nvfp4_rope(t, table, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="y:"):
        nv.nvfp4_rope(t, table, y=t.float())
    cache = nv.KVCache.__new__(nv.KVCache)
    cache.handle, cache.heads, cache.head_dim, cache.buffer = _cache(), 2, 128, torch.zeros(1)
    qa = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    for bad in (dict(lse_out=torch.zeros(3, 4)), dict(slopes=torch.zeros(2)), dict(q_pos=torch.zeros(3)),
                dict(q_doc=torch.zeros(3)), dict(slot_pos=[0])):
        with pytest.raises(ValueError):
            nv.kv_window_attention(cache, [0, 1], [64, 5], qa, 0.1, torch.zeros_like(qa), **bad)
    with pytest.raises(TypeError):
        nv.kv_window_attention(cache, [0], [64], qa.float(), 0.1, torch.zeros_like(qa))
    with pytest.raises(ValueError, match="CUDA"):
        nv.kv_window_attention(cache, [0], [64], qa, 0.1, torch.zeros_like(qa))
    new = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="parents"):
        nv.kv_tree_attention(cache, [0], [64], qa, new, new, torch.zeros(2, dtype=torch.int32), 0.1,
                             torch.zeros_like(qa))
    with pytest.raises(ValueError, match="k_new"):
        nv.kv_tree_attention(cache, [0], [64], qa, new[:2], new, torch.zeros(3, dtype=torch.int32), 0.1,
                             torch.zeros_like(qa))
