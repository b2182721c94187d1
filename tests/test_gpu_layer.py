"""The layer steps on the GPU: RMS norm with NVFP4 output bit for bit against the oracle's
quantization of the FP32 y, rotary positions against binary64."""
import math

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv
import oracle
from gpu_helpers import assert_quant_equal, device_status, mma_padding_is_zero

pytestmark = pytest.mark.gpu


def _bf16(a):
    """float32 -> nearest bf16, as float32."""
    return torch.from_numpy(a).bfloat16().float().numpy()


def norm_reference(x, res, w, eps, bf16):
    """(h, y) in FP32 with the call's roundings.  The root's argument is summed exactly; r has to
    be clear of a rounding border by more than binary64's error for the codes to be decided."""
    h = x if res is None else (x + res).astype(np.float32)
    if bf16 and res is not None:
        h = _bf16(h)
    r = np.empty((len(h), 1), np.float32)
    for i, row in enumerate(h.astype(np.float64)):
        exact = 1.0 / math.sqrt(math.fsum(row * row) / row.size + float(np.float32(eps)))
        lo, hi = exact * (1 - 2.0 ** -47), exact * (1 + 2.0 ** -47)
        assert np.float32(lo) == np.float32(hi), "this input's r is at a rounding border: take another seed"
        r[i] = exact
    y = (h * r).astype(np.float32)
    return h, (y if w is None else (y * w).astype(np.float32))


def run_norm(rows, cols, seed, bf16=True, residual=True, weight="same", given=None, layout=nv.SF_MMA, pad=0, inplace="",
             eps=1e-6, scale=1.0, stream=None):
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if bf16 else torch.float32
    make = lambda s: (lambda a: _bf16(a) if bf16 else a)((rng.standard_normal((rows, cols)) * s).astype(np.float32))
    x, res = make(scale), make(1.0) if residual else None
    x[:, rng.integers(0, cols, max(1, cols // 100))] *= 16.0  # loud channels (a power of two: still bf16)
    wt = {"same": t, "fp32": torch.float32, "bf16": torch.bfloat16, None: None}[weight]
    w = None if wt is None else (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32)
    if wt == torch.bfloat16:
        w = _bf16(w)

    def dev(a):
        big = torch.full((rows, cols + pad), 7.0, dtype=t, device="cuda")
        big[:, :cols] = torch.from_numpy(a).to("cuda", t)
        return big[:, :cols]

    xd, rd = dev(x), dev(res) if residual else None
    wd = None if w is None else torch.from_numpy(w).to("cuda", wt)
    hd = {"": torch.full((rows, cols + pad), 9.0, dtype=t, device="cuda")[:, :cols], "x": xd, "res": rd,
          "none": None}[inplace]
    q = nv.NVFP4Tensor(rows, cols, layout)
    q.codes.fill_(0xEE)
    q.scales.fill_(0xEE)
    g = None if given is None else torch.tensor([given], device="cuda")
    amax = torch.full((1,), -1.0, device="cuda")
    torch.cuda.synchronize()
    nv.nvfp4_rmsnorm_quantize(xd, q, weight=wd, eps=eps, residual=rd, h_out=hd, gscale_in=g, amax_out=amax,
                              stream=stream)
    torch.cuda.synchronize()
    h, y = norm_reference(x, res, w, eps, bf16)
    ref = oracle.quantize(y, gscale=given) if given is not None else oracle.quantize(y)
    assert_quant_equal(q, ref)
    assert amax.item() == np.abs(y).max()
    if layout == nv.SF_MMA:
        assert mma_padding_is_zero(q)
    if hd is not None:
        assert np.array_equal(hd.float().cpu().numpy(), h)
        if pad and hd.stride(0) > cols:  # columns behind the row stay
            whole = torch.as_strided(hd, (rows, cols + pad), (cols + pad, 1))
            assert bool((whole[:, cols:] == (9.0 if inplace == "" else 7.0)).all())
    assert device_status() == nv.OK


# rows of 1, 8 and 9 blocks; the widths where the threads a row change; more blocks than registers keep
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (130, 144), (33, 2048), (5, 2064), (7, 4128), (2, 16400),
                                       (3, 20000), (1, 9216), (300, 512)])
@pytest.mark.parametrize("given", [None, 0.004])
def test_norm_sizes(cuda_dev, rows, cols, given):
    run_norm(rows, cols, rows * 31 + cols, given=given, scale=0.5)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("layout", [nv.SF_MMA, nv.SF_ROWMAJOR])
@pytest.mark.parametrize("residual,inplace", [(True, ""), (True, "x"), (True, "res"), (True, "none"), (False, ""),
                                              (False, "none")])
def test_norm_forms(cuda_dev, bf16, layout, residual, inplace):
    for given in (None, 0.01):
        run_norm(67, 272, 5, bf16=bf16, residual=residual, inplace=inplace, layout=layout, pad=16, given=given)
        run_norm(2, 17008, 6, bf16=bf16, residual=residual, inplace=inplace, layout=layout, pad=16, given=given)


@pytest.mark.parametrize("weight", ["fp32", "bf16", None])
def test_norm_weights(cuda_dev, weight):
    run_norm(9, 1024, 11, bf16=True, weight=weight)
    run_norm(9, 1024, 12, bf16=False, weight=weight, given=0.01)


def test_norm_scales_of_input(cuda_dev):
    """Tiny rows (eps decides), huge rows (the sum needs more than FP32's range), zero rows."""
    run_norm(4, 512, 21, scale=2.0 ** -100, residual=False, eps=1e-12)
    run_norm(4, 512, 22, scale=2.0 ** 80, residual=False)
    run_norm(4, 512, 23, scale=0.0, residual=False)
    run_norm(4, 512, 24, scale=0.0, residual=False, given=0.5, bf16=False)


def test_norm_supplied_scale_saturates(cuda_dev):
    """A scale far too small: block scales stop at 448 and codes at 6, as nvfp4_quantize's do."""
    run_norm(6, 256, 31, given=1e-5)
    run_norm(6, 256, 32, given=0.0)


def test_norm_empty(cuda_dev):
    q = nv.NVFP4Tensor(0, 64)
    g = torch.tensor([0.25], device="cuda")
    amax = torch.full((1,), 3.0, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_rmsnorm_quantize(x, q, gscale_in=g, amax_out=amax)
    assert q.gscale.item() == 0.25 and amax.item() == 0.0
    nv.nvfp4_rmsnorm_quantize(x, q, amax_out=amax)
    assert q.gscale.item() == 0.0 and amax.item() == 0.0


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_norm_nonfinite(cuda_dev, value):
    x = torch.ones(5, 64, dtype=torch.bfloat16, device="cuda")
    x[3, 17] = value
    q = nv.NVFP4Tensor(5, 64)
    q.codes.fill_(0xEE)
    q.scales.fill_(0xEE)
    q.gscale.fill_(5.0)
    nv.nvfp4_rmsnorm_quantize(x, q, amax_out=torch.zeros(1, device="cuda"))
    assert device_status() == nv.ERR_NONFINITE
    assert bool((q.codes == 0xEE).all()) and bool((q.scales == 0xEE).all()) and q.gscale.item() == 5.0
    nv.nvfp4_rmsnorm_quantize(x, q, gscale_in=torch.ones(1, device="cuda"))
    assert device_status() == nv.ERR_NONFINITE
    nv.nvfp4_rmsnorm_quantize(torch.ones_like(x), q, gscale_in=torch.full((1,), math.nan, device="cuda"))
    assert device_status() == nv.ERR_NONFINITE


def test_norm_stream_and_graph(cuda_dev):
    s = torch.cuda.Stream()
    run_norm(40, 512, 41, stream=s)
    # a captured call replayed on new inputs equals the eager one
    x = torch.randn(70, 1024, device="cuda").bfloat16()
    res = torch.randn_like(x)
    h, amax = torch.empty_like(x), torch.zeros(1, device="cuda")
    q, q2 = nv.NVFP4Tensor(70, 1024), nv.NVFP4Tensor(70, 1024)
    h2, amax2 = torch.empty_like(x), torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_rmsnorm_quantize(x, q, residual=res, h_out=h, amax_out=amax)
    for _ in range(3):
        x.copy_(torch.randn_like(x) * 3)
        graph.replay()
        nv.nvfp4_rmsnorm_quantize(x, q2, residual=res, h_out=h2, amax_out=amax2)
        torch.cuda.synchronize()
        assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales) and torch.equal(h, h2)
        assert torch.equal(amax, amax2) and torch.equal(q.gscale, q2.gscale)


# ------------------------------------------------------------------------ rotary positions


def run_rope(n, heads, dim, rot, layout, dtype, pos, table=None, offset=0, pad=0, inplace=False, stream=None):
    """Against binary64.  Each output is one FP32 sum of two products with cosines and sines that
    are within 2^-22 (angle to 2^-23 of a radian, function to 2 ulp, the factor's product), rounded
    to the type: |error| <= 2^-20 (|a| + |b|) m + half a step of the type."""
    gen = torch.Generator().manual_seed(n * 7 + heads)
    flat = torch.randn(n * (heads * dim + pad) + offset, generator=gen).to(dtype).cuda()
    x = torch.as_strided(flat, (n, heads, dim), (heads * dim + pad, dim, 1), offset)
    table = table or nv.RopeTable(rot)
    before, x0 = flat.clone(), x.double().cpu()
    if inplace:
        y = x
    else:
        out = torch.full((n * (heads * dim + pad) + offset,), 5.0, dtype=dtype, device="cuda")
        y = torch.as_strided(out, (n, heads, dim), (heads * dim + pad, dim, 1), offset)
    torch.cuda.synchronize()
    nv.nvfp4_rope(x, table, pos, y=y, layout=layout, stream=stream)
    torch.cuda.synchronize()
    p = pos.double().cpu() if isinstance(pos, torch.Tensor) else torch.arange(n, dtype=torch.float64) + pos
    angle = p[:, None] * table.freq.cpu()
    c, s = torch.cos(angle)[:, None] * table.mscale, torch.sin(angle)[:, None] * table.mscale
    half = rot // 2
    ia, ib = (slice(0, half), slice(half, rot)) if layout == nv.ROPE_HALF else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x0[..., ia], x0[..., ib]
    ref, tol = x0.clone(), torch.zeros_like(x0)
    ref[..., ia], ref[..., ib] = a * c - b * s, a * s + b * c
    tol[..., ia] = tol[..., ib] = 2.0 ** -20 * (a.abs() + b.abs()) * table.mscale
    tol[..., :rot] += torch.finfo(dtype).eps / 2 * (ref.abs() + tol)[..., :rot] + 1e-38
    assert bool(((y.double().cpu() - ref).abs() <= tol).all())
    assert torch.equal(y[..., rot:], before.as_strided(x.shape, x.stride(), offset)[..., rot:])
    if not inplace:
        assert torch.equal(flat, before)
        mask = torch.ones_like(out, dtype=torch.bool)
        torch.as_strided(mask, y.shape, y.stride(), offset).fill_(False)
        assert bool((out[mask] == 5.0).all()), "elements outside the heads were written"
    elif pad:
        mask = torch.ones_like(flat, dtype=torch.bool)
        torch.as_strided(mask, x.shape, x.stride(), offset).fill_(False)
        assert torch.equal(flat[mask], before[mask])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", [nv.ROPE_HALF, nv.ROPE_INTERLEAVED])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n,heads,dim,rot", [(1, 1, 128, 128), (1, 24, 128, 128), (5, 3, 80, 80), (300, 2, 96, 64),
                                             (77, 5, 128, 72), (9, 3, 2, 2), (4, 3, 66, 6), (2, 7, 45, 44),
                                             (3, 2, 4096, 4096), (1025, 24, 64, 16)])
def test_rope_sizes(cuda_dev, dtype, layout, inplace, n, heads, dim, rot):
    run_rope(n, heads, dim, rot, layout, dtype, 17, inplace=inplace, pad=32)


def test_rope_unaligned_and_odd_pitch(cuda_dev):
    for layout in (nv.ROPE_HALF, nv.ROPE_INTERLEAVED):
        for dtype in (torch.bfloat16, torch.float32):
            run_rope(9, 3, 64, 64, layout, dtype, 3, offset=1)
            run_rope(9, 3, 64, 64, layout, dtype, 3, pad=3)


@pytest.mark.parametrize("table", [dict(), dict(scaling="linear", factor=8.0),
                                   dict(base=5e5, scaling="by_parts", factor=16.0, original=4096)])
def test_rope_far_positions(cuda_dev, table):
    t = nv.RopeTable(128, **table)
    pos = torch.tensor([0, 1, 4095, 65537, 999_983, 16_777_217, 2_000_000_011, 2 ** 31 - 1, -5], dtype=torch.int32)
    run_rope(9, 2, 128, 128, nv.ROPE_HALF, torch.float32, pos.cuda(), t)
    run_rope(9, 2, 128, 128, nv.ROPE_HALF, torch.float32, 2 ** 31 - 100, t)


def test_rope_empty_and_stream(cuda_dev):
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_rope(x, nv.RopeTable(64))
    run_rope(33, 4, 64, 64, nv.ROPE_HALF, torch.bfloat16, 5, stream=torch.cuda.Stream())


def test_rope_packed_buffer_into_a_chunk(cuda_dev):
    """q and k rotated in place in a packed q/k/v buffer, and k written straight to a dense chunk."""
    t = nv.RopeTable(128)
    buf = torch.randn(50, 8 + 2 + 2, 128, device="cuda").bfloat16()
    want = buf.clone()
    dense = torch.empty(50, 2, 128, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_rope(buf[:, 8:10], t, 100, y=dense)
    nv.nvfp4_rope(buf[:, :10], t, 100)
    nv.nvfp4_rope(want[:, :8].contiguous(), t, 100)
    assert torch.equal(buf[:, 8:10], dense) and torch.equal(buf[:, 10:], want[:, 10:])


@pytest.mark.parametrize("bf16,cols", [(True, 4112), (True, 14336), (False, 5120)])
@pytest.mark.parametrize("layout", [nv.SF_MMA, nv.SF_ROWMAJOR])
@pytest.mark.parametrize("h,given", [("new", True), ("new", False), ("none", True), ("none", False), ("res", True),
                                     ("res", False)])
def test_norm_many_wide_rows(cuda_dev, bf16, cols, layout, h, given):
    """Several rows a CTA, x and residual by way of shared memory: the same bits as the norm of their
    sum, which takes plain loads."""
    rows = 1203
    dt = torch.bfloat16 if bf16 else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, res = (torch.randn(rows, cols, device="cuda", generator=gen).to(dt) for _ in range(2))
    w = torch.rand(cols, device="cuda", generator=gen).bfloat16()
    g = torch.full((1,), 0.003, device="cuda") if given else None
    total = (x.float() + res.float()).to(dt)
    out = []
    for residual in (None, res.clone()):
        q, amax = nv.NVFP4Tensor(rows, cols, sf_layout=layout), torch.zeros(1, device="cuda")
        q.codes.fill_(0xAA)
        q.scales.fill_(0xAA)
        ho = None
        if residual is not None:
            ho = {"new": torch.empty_like(x), "none": None, "res": residual}[h]
        nv.nvfp4_rmsnorm_quantize(total if residual is None else x, q, weight=w, residual=residual, h_out=ho,
                                  gscale_in=g, amax_out=amax)
        torch.cuda.synchronize()
        out.append((q.codes, q.scales, q.gscale, amax))
    assert device_status() == nv.OK
    assert ho is None or torch.equal(ho, total)
    for want, got in zip(*out):
        assert torch.equal(got, want)
