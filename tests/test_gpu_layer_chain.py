"""The attention half of a decoder layer, as its calls follow one another: RMS norm into NVFP4, the
q/k/v GEMM, rotary positions in the packed buffer, the chunk's append to the cache, attention over
the window (a prefill with causal and sliding masks), then drafted tokens, a decode step and the
output projection.  Each stage is held to binary64 on what the stage before it really produced."""
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
import oracle
from gpu_helpers import assert_quant_equal, device_status
from test_gpu_attention import assert_close, held, reference
from test_gpu_layer import norm_reference

pytestmark = pytest.mark.gpu

HEADS, KV, D, WIDTH = 4, 2, 128, 512


def rotate64(x, pos, table):
    a, b = x[..., :D // 2], x[..., D // 2:]
    t = pos.double()[:, None] * table.freq.cpu()
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def project(x, res, weight, w_qkv, g, h_out):
    """norm -> NVFP4 -> q/k/v in bf16."""
    q = nv.NVFP4Tensor(x.shape[0], WIDTH)
    amax = torch.zeros(1, device="cuda")
    nv.nvfp4_rmsnorm_quantize(x, q, weight=weight, residual=res, h_out=h_out, gscale_in=g, amax_out=amax)
    qkv = torch.empty(x.shape[0], HEADS + 2 * KV, D, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm(q, w_qkv, qkv.view(x.shape[0], -1))
    return q, qkv, amax


def test_layer(cuda_dev):
    gen = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    weight = (1 + 0.1 * rnd(WIDTH)).bfloat16()
    w_qkv, w_o = nv.NVFP4Tensor((HEADS + 2 * KV) * D, WIDTH), nv.NVFP4Tensor(WIDTH, HEADS * D)
    amax = torch.zeros(1, device="cuda")
    nv.nvfp4_quantize((0.05 * rnd(w_qkv.rows, WIDTH)).bfloat16(), w_qkv, amax_out=amax)
    nv.nvfp4_quantize((0.05 * rnd(WIDTH, HEADS * D)).bfloat16(), w_o, amax_out=amax)
    table = nv.RopeTable(D, base=10000.0)
    chunk = 192
    cache = nv.KVCache(KV, D, chunk, 3)
    scale = D ** -0.5
    tokens, k_held, v_held = [], [], []
    g = None
    for n in (192, 77):  # a full chunk, then a partial one
        x, res = rnd(n, WIDTH).bfloat16(), rnd(n, WIDTH).bfloat16()
        x0, res0 = x.float().cpu().numpy(), res.float().cpu().numpy()
        q, qkv, amax = project(x, res, weight, w_qkv, g, res)  # the stream is updated in place
        h, y = norm_reference(x0, res0, weight.float().cpu().numpy(), 1e-6, True)
        assert torch.equal(res.float().cpu(), torch.from_numpy(h))
        assert_quant_equal(q, oracle.quantize(y) if g is None else oracle.quantize(y, gscale=g.item()))
        g = torch.tensor([amax.item() * 1.25 / 2688], device="cuda") if g is None else g
        start = sum(tokens)
        raw = qkv.double().cpu()
        nv.nvfp4_rope(qkv[:, :HEADS + KV], table, start)  # q and k in place, v untouched
        pos = torch.arange(n) + start
        turned = rotate64(raw[:, :HEADS + KV], pos, table)
        spread = raw[:, :HEADS + KV].abs()
        tol = 2.0 ** -19 * (spread + spread.roll(D // 2, -1)) + 2.0 ** -8 * turned.abs() + 2.0 ** -20
        assert bool(((qkv[:, :HEADS + KV].double().cpu() - turned).abs() <= tol).all())
        assert torch.equal(qkv[:, HEADS + KV:].double().cpu(), raw[:, HEADS + KV:])
        k, v = qkv[:, HEADS:HEADS + KV].contiguous(), qkv[:, HEADS + KV:].contiguous()
        nv.kv_quant_append(cache, k, v, len(tokens))
        tokens.append(n)
        kk, vv = held(cache, len(tokens) - 1, n)
        k_held.append(kk)
        v_held.append(vv)
        keys, values = torch.cat(k_held), torch.cat(v_held)
        o = torch.empty(n, HEADS, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(HEADS, n, device="cuda")
        slots = list(range(len(tokens)))
        # q read where it lies in the packed buffer
        nv.kv_window_attention(cache, slots, tokens, qkv[:, :HEADS], scale, o, lse_out=lse, causal=True, window=150,
                               prefix=8, q_pos=start)
        dist = (pos[:, None] - torch.arange(len(keys))[None]).double()
        seen = ((dist >= 0) & (dist < 150)) | (torch.arange(len(keys)) < 8)[None]
        assert_close(o, lse, reference(qkv[:, :HEADS], keys, values, seen, scale))
    # drafts: four continuations of the text and their successors
    parents = torch.tensor([-1, -1, 0, 0, 1, 2, 5], dtype=torch.int32, device="cuda")
    depth = torch.tensor([0, 0, 1, 1, 1, 2, 3])
    n, end = len(parents), sum(tokens)
    _, qkv, _ = project(rnd(n, WIDTH).bfloat16(), None, weight, w_qkv, g, None)
    nv.nvfp4_rope(qkv[:, :HEADS + KV], table, (depth + end).int().cuda())
    o = torch.empty(n, HEADS, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(HEADS, n, device="cuda")
    nv.kv_tree_attention(cache, [0, 1], tokens, qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:], parents,
                         scale, o, lse_out=lse, q_pos=end)
    own = torch.eye(n, dtype=torch.bool)
    for i, p in enumerate(parents.tolist()):
        if p >= 0:
            own[i] |= own[p]
    k_all = torch.cat([keys, qkv[:, HEADS:HEADS + KV].double().cpu()])
    v_all = torch.cat([values, qkv[:, HEADS + KV:].double().cpu()])
    seen = torch.cat([torch.ones(n, len(keys), dtype=torch.bool), own], 1)
    assert_close(o, lse, reference(qkv[:, :HEADS], k_all, v_all, seen, scale))
    # one accepted draft as a decode step of its own gives that draft's row again: the same terms,
    # whose sums may be split otherwise
    one, lse1 = torch.empty_like(o[:1]), torch.empty(HEADS, 1, device="cuda")
    nv.kv_tree_attention(cache, [0, 1], tokens, qkv[:1, :HEADS], qkv[:1, HEADS:HEADS + KV], qkv[:1, HEADS + KV:],
                         parents[:1], scale, one, lse_out=lse1, q_pos=end)
    assert_close(one, lse1, reference(qkv[:1, :HEADS], k_all[:len(keys) + 1], v_all[:len(keys) + 1],
                                      torch.ones(1, len(keys) + 1, dtype=torch.bool), scale))
    # output projection
    qo, out = nv.NVFP4Tensor(n, HEADS * D), torch.empty(n, WIDTH, device="cuda")
    nv.nvfp4_quantize(o.view(n, -1), qo, amax_out=amax)
    nv.nvfp4_gemm(qo, w_o, out)
    a, b = torch.empty(n, HEADS * D, device="cuda"), torch.empty(WIDTH, HEADS * D, device="cuda")
    nv.nvfp4_dequantize(qo, a)
    nv.nvfp4_dequantize(w_o, b)
    bound = a.double().abs() @ b.double().abs().T
    assert bool(((out.double() - a.double() @ b.double().T).abs() <= 1e-5 * bound).all())
    assert device_status() == nv.OK
