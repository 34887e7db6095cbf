"""A kept checkpoint's UE8M0 scales, and the codes for them, are bsmm_quantize's
for every exponent of a block's maximum and on both sides of the significand
1.75, where the scale steps."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ["e4m3", "e5m2"])
def test_scales_at_every_step(code):
    import block_scaled_precision_gemm_gb300 as bsmm
    significands = [0, 1, 0x5FFFFE, 0x5FFFFF, 0x600000, 0x600001, 0x600002, 0x600003, 0x7FFFFF]
    bits = torch.tensor([(e << 23) | s for e in range(255) for s in significands], dtype=torch.int32)
    n = bits.numel()
    g = torch.Generator().manual_seed(1)
    x = (torch.rand(n, 32, generator=g) * 2 - 1) * bits.view(torch.float32)[:, None]
    x[torch.arange(n), torch.arange(n) % 32] = bits.view(torch.float32) * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
    assert bool(torch.isfinite(x).all())
    pad = -n % 128
    x = torch.cat([x, torch.ones(pad, 32)]).view(-1, 64).cuda()  # gate and up: a block each
    want, scales = bsmm.quantize(x, (1, 32), code, "ue8m0")
    _, _, codes, kept = bsmm.gated_act(x, code=code, scale="ue8m0")
    assert torch.equal(kept, scales)
    assert torch.equal(codes, want)
