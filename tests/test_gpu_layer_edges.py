"""The layer steps at uses that go beyond one dense tensor."""
import pytest
import torch

import nvfp4_w4a4_quantized_amax_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [nv.ROPE_HALF, nv.ROPE_INTERLEAVED])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_in_place_in_a_packed_buffer(cuda_dev, layout, dtype):
    """Every rotated head of a packed q/k/v buffer gets what the same heads get in a tensor of their own;
    v stays."""
    t = nv.RopeTable(96)
    buf = torch.randn(50, 8 + 2 + 2, 128, device="cuda").to(dtype)
    was = buf.clone()
    q, k = was[:, :8].contiguous(), was[:, 8:10].contiguous()
    nv.nvfp4_rope(buf[:, :10], t, 100, layout=layout)
    nv.nvfp4_rope(q, t, 100, layout=layout)
    nv.nvfp4_rope(k, t, 100, layout=layout)
    assert torch.equal(buf[:, :8], q) and torch.equal(buf[:, 8:10], k) and torch.equal(buf[:, 10:], was[:, 10:])
    assert not torch.equal(q, was[:, :8])
