"""The operators of a decoder layer around the NVFP4 GEMM and the NVFP4 KV cache: what is
measured, and their plain forms.

  norm   h = x + residual, RMS norm of h, NVFP4 quantization (nvfp4_rmsnorm_quantize)
  rope   rotary positions on a [tokens, heads, head_dim] view of a packed buffer (nvfp4_rope)
  attn   softmax attention of a block of queries over a window of the NVFP4 cache, with a
         tanh cap, a distance bias and causal / sliding / prefix / document masks
         (kv_window_attention)
  tree   attention of a tree of drafted tokens over the cache and over themselves
         (kv_tree_attention)

`own` false computes them from elementary torch operations; true makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
HD = 128  # head_dim of the attention calls
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _norm(name, rows, cols, dtype="bf16", residual=True, given=True):
    return dict(name=name, op="norm", rows=rows, cols=cols, dtype=dtype, residual=residual, given=given)


def _rope(name, tokens, heads, dim, rot, layout, scaling, dtype="bf16", far=0, packed=True):
    return dict(name=name, op="rope", tokens=tokens, heads=heads, dim=dim, rot=rot, layout=layout,
                scaling=scaling, dtype=dtype, far=far, packed=packed)


def _attn(name, tq, kv_heads, group, chunk, fills, cap=0.0, bias=False, causal=False, window=0, prefix=0,
          gap=0, doc_len=0, pad=0):
    return dict(name=name, op="attn", tq=tq, kv_heads=kv_heads, group=group, chunk=chunk, fills=fills, cap=cap,
                bias=bias, causal=causal, window=window, prefix=prefix, gap=gap, doc_len=doc_len, pad=pad)


def _tree(name, drafts, kv_heads, group, chunk, fills, reach, cap=0.0, bias=False):
    return dict(name=name, op="tree", drafts=drafts, kv_heads=kv_heads, group=group, chunk=chunk, fills=fills,
                reach=reach, cap=cap, bias=bias)


def listed():
    return [
        # one decode token before a projection, scale calibrated on earlier tokens
        _norm("norm 1 token", 1, 9216),
        # a chunk of 8192 tokens in the layer's width, residual stream in bf16
        _norm("norm chunk", 8192, 9216),
        # the widest activation with an unknown scale (max|y| first), ragged rows
        _norm("norm unknown scale", 4099, 14336, given=False),
        # one decode token's heads
        _rope("rope 1 token", 1, 24, 128, 128, "half", "none", far=40000),
        # a window's worth of tokens, out of a packed q/k/v buffer, stretched context
        _rope("rope long scaled", 32768, 24, 128, 128, "half", "by_parts", far=1000000),
        # interleaved pairs on part of the head, binary32, odd counts
        _rope("rope part fp32", 8191, 23, 128, 72, "interleaved", "linear", dtype="fp32"),
        # one decode step over four full chunks, one query per cache head
        _attn("attn decode", 1, 24, 1, 8192, "8192,8192,8192,8192"),
        # shared heads, one decode token, short ragged window, distance bias
        _attn("attn shared short", 1, 2, 8, 1024, "1000,77", bias=True, causal=True),
        # a block of queries against the sink-aware window (global sink, shot sink, sliding slots)
        _attn("attn sink window", 1024, 24, 1, 8192, "1024,4096,8192,8192,8192,3000", cap=30.0, causal=True,
              prefix=1024, window=24576, gap=50000),
        # packed documents with shared heads, padded queries behind the last one
        _attn("attn documents", 2000, 4, 4, 4096, "4096,4096,2500", causal=True, doc_len=1500, pad=13),
        # 64 drafted tokens over four full chunks
        _tree("tree 64", 64, 24, 1, 8192, "8192,8192,8192,8192", 9),
        # seven drafts, shared heads, a partial chunk
        _tree("tree 7 shared", 7, 4, 4, 2048, "2048,333", 3, cap=50.0, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _fills(rng, chunk, most):
    """One to six slots, full or partly filled, of `most` tokens in all at the most."""
    got, left = [], most
    for _ in range(rng.randint(1, 6)):
        n = min(chunk if rng.random() < 0.5 else rng.randint(1, chunk), left)
        if n > 0:
            got.append(n)
            left -= n
    return ",".join(map(str, got))


def draw(rng):
    op = rng.choice(("norm", "rope", "attn", "tree"))
    if op == "norm":
        cols = 16 * _log(rng, 8, 896)
        rows = _log(rng, 1, min(8192, 75000000 // cols))
        c = _norm("", rows, cols, rng.choice(("bf16", "bf16", "fp32")), rng.random() < 0.7, rng.random() < 0.5)
    elif op == "rope":
        dim = rng.choice((64, 80, 96, 128, 192, 256))
        rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
        heads = rng.randint(1, 48)
        tokens = _log(rng, 1, min(32768, 100000000 // (heads * dim)))
        c = _rope("", tokens, heads, dim, rot, rng.choice(("half", "interleaved")),
                  rng.choice(("none", "linear", "by_parts")), rng.choice(("bf16", "bf16", "fp32")),
                  rng.choice((0, _log(rng, 1000, 1000000))), rng.random() < 0.5)
    elif op == "attn":
        kv_heads, group = rng.randint(1, 24), rng.choice((1, 1, 2, 4, 8))
        chunk = _log(rng, 64, 8192)
        fills = _fills(rng, chunk, 32768)
        keys = sum(map(int, fills.split(",")))
        tq = _log(rng, 1, max(1, min(2048, 400000000 // (kv_heads * group * keys))))
        causal = rng.random() < 0.5
        c = _attn("", tq, kv_heads, group, chunk, fills, cap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                  bias=rng.random() < 0.3, causal=causal,
                  window=_log(rng, 32, 16384) if rng.random() < 0.3 else 0,
                  prefix=_log(rng, 1, 1024) if causal and rng.random() < 0.4 else 0,
                  gap=rng.choice((0, 0, rng.randint(1, 100000))),
                  doc_len=_log(rng, 50, 4000) if rng.random() < 0.3 else 0, pad=rng.choice((0, 0, 1, 5)))
    else:
        chunk = _log(rng, 64, 8192)
        fills = _fills(rng, chunk, 32768)
        c = _tree("", _log(rng, 1, 128), rng.randint(1, 24), rng.choice((1, 1, 2, 4)), chunk, fills,
                  rng.randint(1, 16), cap=rng.choice((0.0, 0.0, 30.0)), bias=rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- plans


def _ints(text):
    return [int(t) for t in text.split(",")]


def _positions(c):
    """First position of each slot and of the queries: slots follow one another, with a gap
    after the first one; the queries are the window's last tokens."""
    pos, at = [], 0
    for i, n in enumerate(_ints(c["fills"])):
        pos.append(at)
        at += n + (c.get("gap", 0) if i == 0 else 0)
    end = pos[-1] + _ints(c["fills"])[-1]
    if c["op"] == "tree":
        return pos, end
    return pos, max(0, end - c["tq"])


def _rope_args(c):
    """Keyword arguments of the frequency table."""
    if c["scaling"] == "linear":
        return dict(base=10000.0, scaling="linear", factor=4.0)
    if c["scaling"] == "by_parts":
        return dict(base=500000.0, scaling="by_parts", factor=8.0, original=8192, beta_fast=32.0, beta_slow=1.0)
    return dict(base=10000.0, scaling="none")


def _slopes(c):
    n = c["kv_heads"] * c["group"]
    return torch.exp2(-8.0 * torch.arange(1, n + 1, device=DEV, dtype=torch.float32) / n)


def _documents(c):
    """Document of every key and query, by position; the last `pad` queries are in none."""
    pos, q0 = _positions(c)
    kp = torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(pos, _ints(c["fills"]))])
    qp = torch.arange(q0, q0 + c["tq"], device=DEV)
    length = c["doc_len"] or (1 << 40)
    kd, qd = (kp // length).int(), (qp // length).int()
    if c["pad"]:
        qd[-c["pad"]:] = -1
    return kd, qd


# ------------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _align(n):
    return (n + 255) // 256 * 256


def _layout(c):
    """Byte offsets of the cache's parts, as its documentation gives them."""
    slots, width = len(_ints(c["fills"])), c["kv_heads"] * HD
    codes, scales = c["chunk"] * width // 2, c["chunk"] * width // 16
    at, off = 0, {}
    for name, n in (("kc", codes * slots), ("vc", codes * slots), ("ks", scales * slots), ("vs", scales * slots),
                    ("mu", width * 4 * slots), ("g", 8 * slots), ("tokens", 4 * slots)):
        off[name] = at
        at += _align(n)
    off["bytes"], off["codes"], off["scales"] = at, codes, scales
    return off


def _fill_slot(buf, off, slot, k, v, width):
    """One chunk's K (minus its mean) and V in NVFP4, into the cache's bytes."""
    n = k.shape[0]
    mu = k.float().mean(0)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    g = []
    for x, codes_at, scales_at in ((k.float() - mu, "kc", "ks"), (v.float(), "vc", "vs")):
        gs = x.abs().max() / 2688.0
        blocks = x.view(n, width // 16, 16)
        s = (blocks.abs().amax(-1) / (6.0 * gs)).to(torch.float8_e4m3fn)
        d = (s.float() * gs).unsqueeze(-1)
        code = torch.bucketize(blocks.abs() / d.clamp_min(1e-30), mid).to(torch.uint8)
        code = (code + 8 * torch.signbit(blocks).to(torch.uint8)).view(n, width // 2, 2)
        start = off[codes_at] + slot * off["codes"]
        buf[start:start + n * width // 2] = (code[..., 0] | (code[..., 1] << 4)).view(-1)
        start = off[scales_at] + slot * off["scales"]
        buf[start:start + n * width // 16] = s.view(torch.uint8).view(-1)
        g.append(gs)
    start = off["mu"] + slot * width * 4
    buf[start:start + width * 4] = mu.view(torch.uint8).view(-1)
    buf[off["g"] + slot * 8:off["g"] + slot * 8 + 8] = torch.stack(g).view(torch.uint8)
    buf[off["tokens"] + slot * 4:off["tokens"] + slot * 4 + 4] = torch.tensor([n], dtype=torch.int32,
                                                                             device=DEV).view(torch.uint8)


def _cache(c, gen):
    """The bytes of a cache whose K has a mean per (head, dim), as trained keys have."""
    off, heads = _layout(c), c["kv_heads"]
    buf = torch.zeros(off["bytes"], dtype=torch.uint8, device=DEV)
    offset = 3.0 * torch.randn(heads, HD, device=DEV, generator=gen)
    for slot, n in enumerate(_ints(c["fills"])):
        k = torch.randn(n, heads, HD, device=DEV, generator=gen) + offset
        v = torch.randn(n, heads, HD, device=DEV, generator=gen)
        _fill_slot(buf, off, slot, k.bfloat16().view(n, -1), v.bfloat16().view(n, -1), heads * HD)
    return buf, offset


def prepare(case, seed):
    c, gen = dict(case), _gen(seed)
    s = {"c": c}
    if c["op"] == "norm":
        rows, cols, t = c["rows"], c["cols"], DTYPES[c["dtype"]]
        # heavy-tailed activations with some channels thirty times as large
        loud = torch.where(torch.rand(cols, device=DEV, generator=gen) < 0.01, 30.0, 1.0)
        s["x"] = (0.5 * torch.randn(rows, cols, device=DEV, generator=gen) * loud).to(t)
        s["residual"] = torch.randn(rows, cols, device=DEV, generator=gen).to(t) if c["residual"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, device=DEV, generator=gen)).to(t)
        # a scale from earlier calls: a bound on |y| near what these inputs reach
        s["g"] = torch.full((1,), 24.0 / 2688.0, device=DEV) if c["given"] else None
        s["y"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
        s["h"] = torch.empty(rows, cols, dtype=t, device=DEV) if c["residual"] else None
        s["amax"] = torch.empty(1, device=DEV)
        if own:
            import nvfp4_w4a4_quantized_amax_b200 as nv
            s["q"] = nv.NVFP4Tensor(rows, cols)
    elif c["op"] == "rope":
        n, h, d = c["tokens"], c["heads"], c["dim"]
        width = 3 * h if c["packed"] else h
        s["x"] = torch.randn(n, width, d, device=DEV, generator=gen).to(DTYPES[c["dtype"]])[:, width - h:]
        s["y"] = torch.empty(n, h, d, dtype=s["x"].dtype, device=DEV)
        s["pos"] = (torch.arange(n, device=DEV) + c["far"]).int()
        if own:
            import nvfp4_w4a4_quantized_amax_b200 as nv
            s["table"] = nv.RopeTable(c["rot"], **_rope_args(c))
    else:
        heads = c["kv_heads"] * c["group"]
        rows = c["tq"] if c["op"] == "attn" else c["drafts"]
        s["buf"], offset = _cache(c, gen)
        s["q"] = torch.randn(rows, heads, HD, device=DEV, generator=gen).bfloat16()
        s["o"] = torch.empty(rows, heads, HD, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(heads, rows, device=DEV)
        s["slopes"] = _slopes(c) if c["bias"] else None
        s["docs"] = _documents(c) if c["op"] == "attn" and (c["doc_len"] or c["pad"]) else (None, None)
        s["slots"] = list(range(len(_ints(c["fills"]))))
        s["fills"] = _ints(c["fills"])
        s["slot_pos"], s["q_pos"] = _positions(c)
        if c["op"] == "tree":
            k = torch.randn(rows, c["kv_heads"], HD, device=DEV, generator=gen) + offset
            s["k_new"] = k.bfloat16()
            s["v_new"] = torch.randn(rows, c["kv_heads"], HD, device=DEV, generator=gen).bfloat16()
            # each draft continues one of the `reach` drafts before it, or the window itself
            back = (torch.rand(rows, device=DEV, generator=gen) * c["reach"]).int() + 1
            s["parents"] = (torch.arange(rows, device=DEV, dtype=torch.int32) - back).clamp_min(-1).int()
        if own:
            import nvfp4_w4a4_quantized_amax_b200 as nv
            s["cache"] = nv.KVCache(c["kv_heads"], HD, c["chunk"], len(s["slots"]), buffer=s["buf"])
            need = nv.kv_attention_workspace_bytes(s["cache"], s["fills"], rows, heads)
            s["work"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------- the library's calls


def _run_own(s):
    import nvfp4_w4a4_quantized_amax_b200 as nv

    c = s["c"]
    if c["op"] == "norm":
        nv.nvfp4_rmsnorm_quantize(s["x"], s["q"], weight=s["weight"], eps=1e-6, residual=s["residual"], h_out=s["h"],
                                  gscale_in=s["g"], amax_out=s["amax"])
        nv.nvfp4_dequantize(s["q"], s["y"])  # what the 4-bit codes stand for
        return {"y": s["y"], "h": s["h"], "g": s["q"].gscale, "amax": s["amax"]}
    if c["op"] == "rope":
        layout = nv.ROPE_HALF if c["layout"] == "half" else nv.ROPE_INTERLEAVED
        nv.nvfp4_rope(s["x"], s["table"], s["pos"], y=s["y"], layout=layout)
        return s["y"]
    if c["op"] == "attn":
        nv.kv_window_attention(s["cache"], s["slots"], s["fills"], s["q"], HD ** -0.5, s["o"], lse_out=s["lse"],
                               softcap=c["cap"], slopes=s["slopes"], causal=c["causal"], window=c["window"],
                               prefix=c["prefix"], slot_pos=s["slot_pos"], q_pos=s["q_pos"], k_doc=s["docs"][0],
                               q_doc=s["docs"][1], workspace=s["work"])
    else:
        nv.kv_tree_attention(s["cache"], s["slots"], s["fills"], s["q"], s["k_new"], s["v_new"], s["parents"],
                             HD ** -0.5, s["o"], lse_out=s["lse"], softcap=c["cap"], slopes=s["slopes"],
                             slot_pos=s["slot_pos"], q_pos=s["q_pos"], workspace=s["work"])
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------------------ plain forms


def _plain_norm(s):
    c = s["c"]
    x, res = s["x"], s["residual"]
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    # the sum of squares of a long row in 64 bits: the codes next to a border go by its last bits
    eps = torch.tensor(1e-6, dtype=torch.float32, device=DEV).double()
    r = (1.0 / torch.sqrt(h.double().square().sum(-1, keepdim=True) / c["cols"] + eps)).float()
    y = (h.float() * r) * s["weight"].float()
    amax = y.abs().max().view(1)
    g = s["g"] if c["given"] else amax / torch.full((1,), 2688.0, device=DEV)
    blocks = y.view(c["rows"], c["cols"] // 16, 16)
    ratio = blocks.abs().amax(-1) / (g * 6.0)
    sc = ratio.clamp_max(448.0).to(torch.float8_e4m3fn).float()
    a = blocks.abs().double()
    d = (sc * g).double().unsqueeze(-1)
    # nearest of the eight magnitudes, ties to the even one: two products decide each border exactly
    m = 0.5 * ((a > 0.25 * d).float() + (a >= 0.75 * d).float() + (a > 1.25 * d).float() + (a >= 1.75 * d).float())
    m = m + (a > 2.5 * d).float() + (a >= 3.5 * d).float() + 2.0 * (a > 5.0 * d).float()
    m = torch.where(d > 0, m, torch.zeros_like(m))
    v = torch.copysign(m, blocks) * sc.unsqueeze(-1) * g
    return {"y": v.view(c["rows"], c["cols"]).to(torch.bfloat16), "h": None if res is None else h, "g": g,
            "amax": amax}


def _frequencies(c):
    """Rotation per position of each pair, in 64 bits, and the factor on cos and sin."""
    a, rot = _rope_args(c), c["rot"]
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    f = a["base"] ** (-2.0 * i / rot)
    if a["scaling"] == "linear":
        return f / a["factor"], 1.0
    if a["scaling"] == "by_parts":
        # interpolation by parts (Peng et al. 2023): pairs that turn often keep their frequency,
        # pairs that turn seldom are stretched by the factor, with a ramp between them
        at = [rot * math.log(a["original"] / (b * 2 * math.pi)) / (2 * math.log(a["base"]))
              for b in (a["beta_fast"], a["beta_slow"])]
        lo, hi = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f / a["factor"] * ramp + f * (1.0 - ramp), 0.1 * math.log(a["factor"]) + 1.0
    return f, 1.0


def _plain_rope(s):
    c, x = s["c"], s["x"].float()
    rot = c["rot"]
    f, m = _frequencies(c)
    angle = s["pos"].double()[:, None] * f  # 64 bits: far positions turn many times
    cos, sin = (torch.cos(angle) * m).float()[:, None], (torch.sin(angle) * m).float()[:, None]
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1).to(s["x"].dtype)


def _decoded(s):
    """K^ and V^ of the window's keys, [kv_heads, keys, 128], binary32 (every slot is as long
    as the case's chunk: the rows behind a slot's last token are dropped)."""
    c, off, buf = s["c"], _layout(s["c"]), s["buf"]
    n, heads, chunk = len(s["slots"]), c["kv_heads"], c["chunk"]
    width = heads * HD
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    keep = torch.arange(chunk, device=DEV)[None] < torch.tensor(s["fills"], device=DEV)[:, None]
    mu = buf[off["mu"]:off["mu"] + n * width * 4].view(torch.float32).view(n, 1, heads, HD)
    g = buf[off["g"]:off["g"] + 8 * n].view(torch.float32).view(n, 2, 1, 1, 1)

    def part(codes_at, scales_at, gs, mean):
        b = buf[off[codes_at]:off[codes_at] + n * off["codes"]].view(n, chunk, heads, HD // 2)
        e = torch.stack([lut[(b & 15).long()], lut[(b >> 4).long()]], -1).view(n, chunk, heads, HD // 16, 16)
        sc = buf[off[scales_at]:off[scales_at] + n * off["scales"]].view(torch.float8_e4m3fn)
        v = (e * sc.float().view(n, chunk, heads, HD // 16, 1)).view(n, chunk, heads, HD) * gs
        v = v if mean is None else v + mean
        return v[keep].transpose(0, 1)

    return part("kc", "ks", g[:, 0], mu), part("vc", "vs", g[:, 1], None)


def _visible(c, kp, qp, kd, qd):
    """Which keys each query sees, [queries, keys]."""
    d = qp[:, None] - kp[None]
    ok = torch.ones_like(d, dtype=torch.bool)
    if c.get("causal"):
        ok = ok & (d >= 0)
    if c.get("window"):
        ok = ok & (d < c["window"])
    if c.get("prefix"):
        ok = ok | (kp < c["prefix"])[None]
    if kd is not None:
        ok = ok & (qd[:, None] == kd[None])
    return ok


def _key_positions(s):
    return torch.cat([torch.arange(p, p + n, device=DEV) for p, n in zip(s["slot_pos"], s["fills"])])


def _scores(s, q, k, distance):
    """Capped and biased scores [kv_heads, group * rows, keys] of q [kv_heads, group * rows, 128]."""
    c = s["c"]
    x = torch.matmul(q, k.transpose(1, 2)) * (HD ** -0.5)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["bias"]:
        h, rows = c["kv_heads"], distance.shape[0]
        x = x.view(h, c["group"], rows, -1) - s["slopes"].view(h, -1, 1, 1) * distance.abs().float()
        x = x.view(h, c["group"] * rows, -1)
    return x


def _grouped(s, q):
    """[rows, heads, 128] -> [kv_heads, group * rows, 128]."""
    c = s["c"]
    return q.float().view(-1, c["kv_heads"], c["group"], HD).permute(1, 2, 0, 3).reshape(c["kv_heads"], -1, HD)


def _attend(s, x, seen, v):
    """Softmax of the visible scores x and its sum over v; a row that sees nothing gives 0 and -inf."""
    c = s["c"]
    rows, h, group = seen.shape[0], c["kv_heads"], c["group"]
    x = x.view(h, group, rows, -1).masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(h, group * rows, -1), v).view(h, group, rows, HD)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + torch.log(total)).view(h * group, rows)
    return {"o": o.permute(2, 0, 1, 3).reshape(rows, h * group, HD).to(torch.bfloat16), "lse": lse}


def _plain_attn(s):
    c = s["c"]
    k, v = _decoded(s)
    kp = _key_positions(s)
    qp = torch.arange(s["q_pos"], s["q_pos"] + c["tq"], device=DEV)
    kd, qd = s["docs"]
    x = _scores(s, _grouped(s, s["q"]), k, qp[:, None] - kp[None])
    return _attend(s, x, _visible(c, kp, qp, kd, qd), v)


def _ancestors(parents):
    """[i, j]: whether draft j is i or one of its ancestors (closure of the parent relation)."""
    n = parents.numel()
    j = torch.arange(n, device=DEV)
    a = ((parents[:, None] == j[None]) | (j[:, None] == j[None])).float()
    for _ in range(max(1, n).bit_length()):
        a = (torch.matmul(a, a) > 0).float()
    return a > 0


def _plain_tree(s):
    c = s["c"]
    k, v = _decoded(s)
    a = _ancestors(s["parents"])
    depth = a.sum(-1) - 1
    qp = s["q_pos"] + depth
    kp = torch.cat([_key_positions(s), qp])
    k = torch.cat([k, s["k_new"].float().transpose(0, 1)], 1)
    v = torch.cat([v, s["v_new"].float().transpose(0, 1)], 1)
    seen = torch.cat([torch.ones(a.shape[0], sum(s["fills"]), dtype=torch.bool, device=DEV), a], 1)
    x = _scores(s, _grouped(s, s["q"]), k, qp[:, None] - kp[None])
    return _attend(s, x, seen, v)


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn, "tree": _plain_tree}[state["c"]["op"]](state)


# ------------------------------------------------------------------------------------- work


def _pairs(c):
    """Visible (query, key) pairs of one head."""
    pos, q0 = _positions(c)
    fills = _ints(c["fills"])
    if c["op"] == "tree":  # ancestors are few next to the window
        return c["drafts"] * (sum(fills) + 1)
    kp = np.concatenate([np.arange(p, p + n) for p, n in zip(pos, fills)])
    length, total = c["doc_len"], 0
    for i in range(c["tq"] - c["pad"]):
        d = q0 + i - kp
        ok = np.ones(kp.size, bool)
        if c["causal"]:
            ok &= d >= 0
        if c["window"]:
            ok &= d < c["window"]
        if c["prefix"]:
            ok |= kp < c["prefix"]
        if length:
            ok &= kp // length == (q0 + i) // length
        total += int(ok.sum())
    return total


def work(case):
    c = case
    if c["op"] == "norm":
        n, size = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        # x (and the residual) read; the stream, the codes with their scales and the values written
        return {"bytes": n * (size * (3 if c["residual"] else 1) + 0.5625 + 2) + c["cols"] * size, "flops": 12.0 * n}
    if c["op"] == "rope":
        n, size = c["tokens"] * c["heads"] * c["dim"], 2 if c["dtype"] == "bf16" else 4
        return {"bytes": 2.0 * n * size + 4 * c["tokens"], "flops": 3.0 * n * c["rot"] / c["dim"]}
    heads = c["kv_heads"] * c["group"]
    rows = c["tq"] if c["op"] == "attn" else c["drafts"]
    keys = sum(_ints(c["fills"]))
    b = keys * c["kv_heads"] * HD * 2 * 0.5625 + rows * heads * (HD * 4 + 4)
    if c["op"] == "tree":
        b += rows * c["kv_heads"] * HD * 4
    return {"bytes": float(b), "flops": 4.0 * HD * heads * max(1, _pairs(c))}


# ------------------------------------------------------------------------------------ 64 bits


def _quantized64(y, g):
    """What NVFP4 with tensor scale g (binary32) holds of y, from the format's definition."""
    rows, cols = y.shape
    b = y.reshape(rows, cols // 16, 16)
    top = b.abs().amax(2)
    ratio = top / (6.0 * g)
    s = torch.minimum(ratio, torch.full_like(ratio, 448.0)).float().to(torch.float8_e4m3fn).double()
    step = (s * g)[..., None]
    t = b.abs() / torch.where(step > 0, step, torch.ones_like(step))
    # spacing 0.5 below 2, 1 below 4, 2 above; round() takes ties to even, as the codes do
    t = torch.where(t < 1.75, torch.round(t * 2) / 2, torch.where(t < 3.5, torch.round(t), torch.round(t / 2) * 2))
    t = torch.where(step > 0, t.clamp(max=6.0), torch.zeros_like(t))
    return (torch.sign(b) * t * step).reshape(rows, cols)


def _exact_norm(s):
    c = s["c"]
    h = s["x"].double()
    out_h = None
    if s["residual"] is not None:
        out_h = h + s["residual"].double()
        h = out_h.to(s["x"].dtype).double()
    eps = float(np.float32(1e-6))
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * s["weight"].double()
    amax = y.abs().max()
    g = s["g"].double()[0] if c["given"] else (amax / 2688.0).float().double()
    return {"y": _quantized64(y, g), "h": out_h, "g": g.view(1), "amax": amax.view(1)}


def _exact_rope(s):
    c = s["c"]
    a, rot = _rope_args(c), c["rot"]
    f = np.exp(-np.log(a["base"]) * np.arange(0, rot, 2) / rot)
    m = 1.0
    if a["scaling"] == "linear":
        f = f / a["factor"]
    elif a["scaling"] == "by_parts":
        # turns over the original length: beta_fast and more keep f, beta_slow and fewer take f / factor,
        # with whole pair numbers as the ends of the ramp
        ends = [rot / 2 * np.log(a["original"] / (2 * np.pi * b)) / np.log(a["base"])
                for b in (a["beta_fast"], a["beta_slow"])]
        lo, hi = max(0.0, np.floor(ends[0])), min(rot - 1.0, np.ceil(ends[1]))
        mix = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        f = f * (1 - mix + mix / a["factor"])
        m = 1.0 + 0.1 * np.log(a["factor"])
    f = torch.tensor(f, device=DEV)
    x = s["x"].double()
    half = c["rot"] // 2
    z = torch.polar(torch.full((c["tokens"], half), m, dtype=torch.float64, device=DEV), s["pos"].double()[:, None] * f)
    out = x.clone()
    if c["layout"] == "half":
        w = torch.complex(x[..., :half], x[..., half:2 * half]) * z[:, None]
        out[..., :half], out[..., half:2 * half] = w.real, w.imag
    else:
        w = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * z[:, None]
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = w.real, w.imag
    return out


def _exact_keys(s, head):
    """K^ and V^ of one cache head, [keys, 128], 64 bits, slot by slot from the bytes."""
    c, off, buf = s["c"], _layout(s["c"]), s["buf"]
    heads = c["kv_heads"]
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    ks, vs = [], []
    for slot, n in zip(s["slots"], s["fills"]):
        g = buf[off["g"] + 8 * slot:off["g"] + 8 * slot + 8].view(torch.float32).double()
        mu = buf[off["mu"] + slot * heads * HD * 4:][:heads * HD * 4].view(torch.float32).view(heads, HD)[head].double()
        for to, codes_at, scales_at, gs, mean in ((ks, "kc", "ks", g[0], mu), (vs, "vc", "vs", g[1], 0.0)):
            b = buf[off[codes_at] + slot * off["codes"]:][:n * heads * HD // 2].view(n, heads, HD // 2)[:, head]
            nib = torch.stack([b % 16, b // 16], 2).reshape(n, HD).long()
            val = table[nib % 8] * torch.where(nib >= 8, -1.0, 1.0)
            sc = buf[off[scales_at] + slot * off["scales"]:][:n * heads * HD // 16].view(n, heads, HD // 16)[:, head]
            sc = sc.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
            to.append(val * sc * gs + mean)
    return torch.cat(ks), torch.cat(vs)


def _exact_attention(s):
    c = s["c"]
    heads, group = c["kv_heads"] * c["group"], c["group"]
    rows = s["q"].shape[0]
    o = torch.zeros(rows, heads, HD, dtype=torch.float64, device=DEV)
    lse = torch.zeros(heads, rows, dtype=torch.float64, device=DEV)
    kp = _key_positions(s)
    if c["op"] == "tree":
        parents = s["parents"].tolist()
        depth, anc = [], torch.zeros(rows, rows, dtype=torch.bool)
        for i, p in enumerate(parents):
            depth.append(0 if p < 0 else depth[p] + 1)
            if p >= 0:
                anc[i] = anc[p]
            anc[i, i] = True
        qp = s["q_pos"] + torch.tensor(depth, device=DEV)
        seen = torch.cat([torch.ones(rows, kp.numel(), dtype=torch.bool, device=DEV), anc.to(DEV)], 1)
        kp = torch.cat([kp, qp])
    else:
        qp = torch.arange(rows, device=DEV) + s["q_pos"]
        seen = _visible(c, kp, qp, *s["docs"])
    away = (qp[:, None] - kp[None]).abs().double()
    for head in range(heads):
        if head % group == 0:
            k, v = _exact_keys(s, head // group)
            if c["op"] == "tree":
                k = torch.cat([k, s["k_new"][:, head // group].double()])
                v = torch.cat([v, s["v_new"][:, head // group].double()])
        x = s["q"][:, head].double() @ k.T / math.sqrt(HD)
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        if c["bias"]:
            x = x - s["slopes"][head].double() * away
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        lse[head] = torch.logsumexp(x, 1)
        p = torch.exp(x - torch.where(torch.isinf(lse[head]), torch.zeros_like(lse[head]), lse[head])[:, None])
        o[:, head] = p @ v
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attention, "tree": _exact_attention}[case["op"]](s)
