"""One row of more than 2^27 columns (backward) or 2^28 (forward): the same codes,
scales and results as its pieces as rows of their own."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def test_backward_of_a_very_wide_row():
    bsmm = _bsmm()
    n, I = 64, 2 ** 27 + 2 ** 20  # 64 pieces
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(-127, 128, (n, 2 * I // n), dtype=torch.int8, device="cuda", generator=g)
    scales = torch.rand(n, 2 * I // n // 128, device="cuda", generator=g) * 0.05
    dh = torch.randn(n, I // n, device="cuda", generator=g).bfloat16()
    ref, href = bsmm.gated_act_backward(dh, codes, scales, return_h=True)

    def wide(t):  # [n, gate | up] -> [1, gate | up]
        gate, up = t.chunk(2, dim=1)
        return torch.cat([gate.reshape(1, -1), up.reshape(1, -1)], 1)

    d, h = bsmm.gated_act_backward(dh.view(1, -1), wide(codes), wide(scales), return_h=True)
    assert torch.equal(h.view(-1), href.view(-1))
    assert torch.equal(d, wide(ref))


def test_forward_of_a_very_wide_row():
    bsmm = _bsmm()
    n, I = 64, 2 ** 28 + 2 ** 20
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.empty(n, 2 * I // n, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ref = bsmm.gated_act(x, code="e4m3", scale="ue8m0")
    gate, up = x.chunk(2, dim=1)
    got = bsmm.gated_act(torch.cat([gate.reshape(1, -1), up.reshape(1, -1)], 1), code="e4m3", scale="ue8m0")
    for k in (0, 1):
        assert torch.equal(got[k].view(-1), ref[k].view(-1))
    for k in (2, 3):
        a, b = ref[k].chunk(2, dim=1)
        assert torch.equal(got[k][0], torch.cat([a.reshape(-1), b.reshape(-1)]))
