"""bsmm_gated_act and its backward where the activation nearly vanishes or is
nearly the identity: relative errors, with no absolute allowance but what
binary32's smallest numbers need.

SiLU and GELU and both terms of their derivatives (p and g p (1 - p), Phi and g
times the density) are each held to 2^-20 of themselves: exp to 2^-22, a
reciprocal or erfc to 2^-22, three roundings.  Products with dh and u add three
roundings of 2^-24.  An activation below 2^-126 is a multiple of 2^-149."""

import numpy as np
import pytest
import torch

from oracle import formats as F

pytestmark = pytest.mark.gpu

REL = 2.0 ** -20 + 2.0 ** -22
TINY = 2.0 ** -148  # of a subnormal act, times the factor after it, or of a subnormal result


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def act64(g, act):
    """act(g) and the two terms of its derivative, on float64 tensors."""
    if act == "silu":
        p = torch.exp(torch.clamp(g, max=0)) / (1 + torch.exp(-g.abs()))
        q = torch.exp(torch.clamp(-g, max=0)) / (1 + torch.exp(-g.abs()))  # 1 - p
        return g * p, p, g * p * q
    cdf = 0.5 * torch.special.erfc(-g * 0.5 ** 0.5)
    return g * cdf, cdf, g * torch.exp(-0.5 * g * g) * (2 * np.pi) ** -0.5


def inside(got, ref, tol, what):
    spacing = 2.0 ** -133 if got.dtype == torch.bfloat16 else 0.0
    bad = ~(((got.double() - ref).abs() <= tol + spacing / 2) | (got.double() == ref))  # (infinities are equal)
    assert not bad.any(), (what, int(bad.sum()), [float(v[bad].flatten()[0]) for v in (got.double(), ref, tol)])


@pytest.mark.parametrize("act,largest", [("silu", [1, 4, 10, 20, 40, 60, 79, 81, 86, 90, 100, 130, 1e4]),
                                         ("gelu", [1, 2, 4, 8, 10, 12, 13, 14, 20, 100, 1e20])])
@pytest.mark.parametrize("fmt", ["int8", "e4m3 f32", "e4m3 ue8m0", "e5m2 ue8m0"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(act, largest, fmt, dtype):
    bsmm = _bsmm()
    code, scale = (fmt.split() + ["f32"])[:2]
    I, rows = 1024, 8
    M = rows * len(largest)
    g = torch.Generator().manual_seed(len(largest))
    block = 128 if scale == "f32" else 32
    if code == "int8":
        codes = torch.randint(-127, 128, (M, 2 * I), generator=g, dtype=torch.int16).to(torch.int8)
        values, qmax = codes.double(), 127.0
    else:
        codes = torch.randint(0, 256, (M, 2 * I), generator=g, dtype=torch.int16).to(torch.uint8)
        codes[(codes & 0x7F) >= (0x7F if code == "e4m3" else 0x7C)] = 0x38
        values, qmax = torch.from_numpy(F.decode(codes.numpy(), code).astype(np.float64)), 448.0 if code == "e4m3" else 57344.0
    top = torch.tensor(largest, dtype=torch.float64).repeat_interleave(rows)[:, None].expand(M, I // block)
    s = torch.cat([top / qmax, torch.full((M, I // block), 3.0 / qmax, dtype=torch.float64)], 1).float()
    if scale == "ue8m0":
        stored = (torch.log2(s).ceil() + 127).clamp(0, 254).to(torch.uint8)
        s = torch.exp2(stored.float() - 127)
    else:
        stored = s
    v = (values.view(M, -1, block) * s.double()[..., None]).float().view(M, 2 * I).double()
    gate, up = v[:, :I], v[:, I:]
    dh = torch.randn(M, I, generator=g).to(dtype)
    d, h = bsmm.gated_act_backward(dh.cuda(), codes.cuda(), stored.cuda(), act=act, code=code, scale=scale, return_h=True)
    f, a, b = act64(gate, act)
    w, wu = dh.double(), dh.double() * up
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    out = d.cpu()
    ref = w * f
    inside(out[:, I:], ref, (REL + half) * ref.abs() + TINY * (1 + w.abs()), "d_up")
    ref = wu * (a + b)
    inside(out[:, :I], ref, REL * wu.abs() * (a.abs() + b.abs()) + half * ref.abs() + TINY * (1 + wu.abs()), "d_gate")
    ref = f * up
    inside(h.cpu(), ref, (REL + 2.0 ** -8) * ref.abs() + TINY * (1 + up.abs()), "h")


@pytest.mark.parametrize("code,scale", [(None, "f32"), ("int8", "f32"), ("e4m3", "ue8m0")])
@pytest.mark.parametrize("act,low,high", [("silu", -102.0, -60.0), ("silu", -12.0, 110.0), ("gelu", -13.5, -8.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_forward(act, low, high, code, scale, dtype):
    """h of vanishing activations times large numbers."""
    bsmm = _bsmm()
    M, I = 5, 4096
    gate = torch.linspace(low, high, I).expand(M, I)
    up = 1e30 * (1 + torch.rand(M, I, generator=torch.Generator().manual_seed(2)))
    x = torch.cat([gate, up], 1).to(dtype)
    f = act64(x[:, :I].double(), act)[0]
    ref, tiny = f * x[:, I:].double(), TINY * (1 + x[:, I:].double().abs())
    h, _, _, _ = bsmm.gated_act(x.cuda(), act=act, h_type="bf16", code=code, scale=scale)
    inside(h.cpu(), ref, (2.0 ** -8 + 2.0 ** -15) * ref.abs() + tiny, "bf16")
    # E4M3: half a unit of 3 bits; a block's maximum is 256 times its smallest normal code at least
    q, qs, _, _ = bsmm.gated_act(x.cuda(), act=act, h_type="e4m3", code=code, scale=scale)
    s = torch.exp2(qs.cpu().double() - 127).repeat_interleave(32, 1)
    got = torch.from_numpy(F.decode(q.cpu().numpy(), "e4m3").astype(np.float64)) * s
    inside(got, ref, 2.0 ** -4 * (1 + 2.0 ** -12) * ref.abs() + tiny + s * 2.0 ** -10, "e4m3")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_numbers(act, dtype):
    """Gates up to bfloat16's largest magnitude, as masks write them, and the
    infinities that an E4M3 checkpoint makes of the largest: zero below, the
    identity above, forward and backward, beside ordinary numbers."""
    bsmm = _bsmm()
    top = (2 - 2.0 ** -7) * 2.0 ** 127
    special = torch.tensor([-top, -2.5e38, -2.3e38, -1e38, -1e20, -600.0, top, 2.5e38, 2.3e38, 1e38, 1e20, 600.0])
    I = 32 * len(special)
    gate = torch.randn(4, len(special), 32, generator=torch.Generator().manual_seed(3))
    gate[:, :, 7] = special
    gate = gate.view(4, I).to(dtype)
    up = torch.full((4, I), 0.5).to(dtype)
    f = act64(gate.double(), act)[0]
    f[gate < -500] = 0
    f[gate > 500] = gate[gate > 500].double()
    x = torch.cat([gate, up], 1).cuda()
    for code, scale in ((None, "f32"), ("int8", "f32"), ("e4m3", "ue8m0")):
        h, _, codes, scales = bsmm.gated_act(x, act=act, h_type="bf16", code=code, scale=scale)
        inside(h.cpu(), f * 0.5, (2.0 ** -8 + 2.0 ** -15) * (f * 0.5).abs() + TINY, "h")
    # every block has one of them: in the checkpoint they stand beside zeros
    dh = torch.full((4, I), 0.25, device="cuda").to(dtype)
    d, h = bsmm.gated_act_backward(dh, codes, scales, act=act, code=code, scale=scale, return_h=True)
    v = torch.from_numpy(F.decode(codes.cpu().numpy(), code).astype(np.float64)).view(4, -1, 32)
    v = (v * torch.exp2(scales.cpu().double() - 127)[..., None]).view(4, 2 * I).float().double()
    assert bool(v.isinf().any())  # E4M3 rounds the largest numbers up to 2^128
    g, u = v[:, :I], v[:, I:]
    big = g.abs() > 500
    small = torch.where(big, torch.zeros_like(g), g)
    f, p, q = act64(small, act)
    f = torch.where(big, g.clamp(min=0), f)
    slope, terms = (torch.where(big, (g > 0).double(), t) for t in (p + q, p.abs() + q.abs()))
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    out = d.cpu()
    inside(out[:, I:], 0.25 * f, (REL + half) * (0.25 * f).abs() + TINY, "d_up")
    inside(out[:, :I], 0.25 * u * slope, 0.25 * u * (REL * terms + half * slope.abs()) + TINY, "d_gate")
    inside(h.cpu(), f * u, (REL + 2.0 ** -8) * (f * u).abs() + TINY, "h again")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("largest", [1.0, 300.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_stays_where_it_is(act, largest, dtype):
    """A NaN gate or up gives NaN in its own place and nowhere else, beside large
    numbers or not; so does a NaN code of a checkpoint."""
    bsmm = _bsmm()
    M, I = 3, 256
    g = torch.Generator().manual_seed(4)
    x = torch.rand(M, 2 * I, generator=g).to(dtype)
    x[:, ::32] = largest
    x[0, 5], x[1, 70], x[2, I + 9] = float("nan"), float("nan"), float("nan")
    want = torch.zeros(M, I, dtype=torch.bool)
    want[0, 5] = want[1, 70] = want[2, 9] = True
    for code, scale in ((None, "f32"), ("int8", "f32"), ("e5m2", "ue8m0")):
        h, _, _, _ = bsmm.gated_act(x.cuda(), act=act, h_type="bf16", code=code, scale=scale)
        assert torch.equal(h.isnan().cpu(), want), code
    clean = torch.nan_to_num(x.float(), nan=0.25).to(dtype)
    _, _, codes, scales = bsmm.gated_act(clean.cuda(), act=act, code="e4m3", scale="ue8m0")
    codes[0, 5], codes[1, 70], codes[2, I + 9] = 0x7F, 0x7F, 0x7F
    dh = torch.rand(M, I, generator=g).to(dtype) + 0.5
    d, h = bsmm.gated_act_backward(dh.cuda(), codes, scales, act=act, code="e4m3", scale="ue8m0", return_h=True)
    assert torch.equal(h.isnan().cpu(), want)
    nan = d.isnan().cpu()
    assert torch.equal(nan[:, :I], want)  # d_gate takes both
    want[2, 9] = False
    assert torch.equal(nan[:, I:], want)  # d_up takes the gate
