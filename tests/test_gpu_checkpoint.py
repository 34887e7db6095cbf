"""bsmm_gated_act, bsmm_gated_act_backward and bsmm_linear_backward_checkpoint.

Checkpoint codes and scales are compared bit for bit.  h and the gradients are
computed in binary32 with exp and a division good to 2 ulp: every value is
within 2^-20 of its magnitude (a few operations of at most 2^-22 each, the
exponent's argument adding |g| 2^-24), before the rounding of its type, where
the magnitude of a gradient of gate counts both terms of act'."""

import numpy as np
import pytest
import torch

from oracle import checkpoint as O
from oracle import formats as F
from oracle import gemm as G

from test_gpu_atoms import decode_atoms

pytestmark = pytest.mark.gpu

FORMATS = [("int8", "f32"), ("e4m3", "f32"), ("e5m2", "f32"), ("e4m3", "ue8m0"), ("e5m2", "ue8m0")]
REL = 2.0 ** -20


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def gate_up(M, I, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed * 101 + M * 7 + I)
    x = torch.randn(M, 2 * I, generator=g) * 1.5
    x[0, :32] = 0                      # all-zero blocks
    if M > 1:
        x[1, :] = 0
        x[M - 1, I:I + 64] = -0.0
    if M > 2:
        x[2, :I] = torch.linspace(-30, 30, I)  # saturated and vanishing activations
        x[2, 5] = 448.0 * 4           # a block whose maximum is a code times a power of two
    return x.to(dtype)


@pytest.mark.parametrize("code,scale", FORMATS + [(None, "f32")])
@pytest.mark.parametrize("M,I,act,dtype", [(1, 128, "silu", torch.bfloat16), (3, 384, "gelu", torch.bfloat16),
                                           (37, 256, "silu", torch.float32), (130, 1024, "gelu", torch.float32),
                                           (1001, 640, "silu", torch.bfloat16)])
def test_forward(M, I, act, dtype, code, scale):
    bsmm = _bsmm()
    x = gate_up(M, I, 1, dtype)
    xf = x.float().numpy()
    # h is a binary32 number: what is too small for one is a zero, and a block of those an all-zero block
    ref = O.gated(xf, act).astype(np.float32).astype(np.float64)
    tol = REL * np.abs(ref) + 1e-37
    h, hs, codes, scales = bsmm.gated_act(x.cuda(), act=act, h_type="bf16", code=code, scale=scale)
    assert hs is None and h.dtype == torch.bfloat16
    got = h.float().cpu().numpy()
    assert (np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref)).all()
    if code is None:
        assert codes is None and scales is None
    else:
        oc, os_ = O.keep(xf, code, scale)
        np.testing.assert_array_equal(codes.cpu().numpy(), oc)
        np.testing.assert_array_equal(scales.cpu().numpy(), os_)
    for ht in ("e4m3", "e5m2"):
        q, qs, c2, s2 = bsmm.gated_act(x.cuda(), act=act, h_type=ht, code=code, scale=scale)
        if code is not None:
            assert torch.equal(c2, codes) and torch.equal(s2, scales)
        e = qs.cpu().numpy().astype(np.int64) - 127
        amax = np.abs(ref).reshape(M, I // 32, 32).max(-1)
        # the exponent: that of a maximum within REL of the reference's
        lo, hi = (O.ue8m0_exponent(amax * f, ht) for f in (1 - REL, 1 + REL))
        assert ((e >= lo) & (e <= hi)).all()
        s = np.exp2(e.astype(np.float64)).repeat(32, axis=1)
        v = F.decode(q.cpu().numpy(), ht).astype(np.float64)
        # half a step of the code grid at the quotient, or of the finer binade below a power of two
        bits, low = (3, -6) if ht == "e4m3" else (2, -14)
        r = np.abs(ref) / s
        step = np.exp2(np.floor(np.log2(np.maximum(r * (1 + REL), 2.0 ** low))) - bits)
        assert (np.abs(v - ref / s) <= step / 2 + 2 * REL * r + 1e-30).all()


def test_forward_layouts():
    """Strided gate_up, and h's scales in the atom layout (with padding)."""
    bsmm = _bsmm()
    M, I = 150, 160
    x = gate_up(M, I, 3).cuda()
    q, qs, _, _ = bsmm.gated_act(x, code=None)
    atoms = bsmm.gated_act(x, code=None, h_scales_are_atoms=True)
    assert torch.equal(atoms[0], q)
    np.testing.assert_array_equal(decode_atoms(atoms[1].cpu().numpy(), 1, M, I, "mxfp8")[0], qs.cpu().numpy())
    wide = torch.full((M, 2 * I + 48), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 2 * I] = x
    h = torch.empty((M, I), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, I // 32), dtype=torch.uint8, device="cuda")
    L, P = bsmm.lib(), bsmm._ptr
    assert L.bsmm_gated_act(P(wide[:, 8:]), bsmm.BF16, M, I, 2 * I + 48, bsmm.SILU, bsmm.E4M3, P(h), P(s), 0, 0, 0, None,
                            None, bsmm._stream()) == bsmm.OK
    assert torch.equal(h, q) and torch.equal(s, qs)


@pytest.mark.parametrize("code,scale", FORMATS)
@pytest.mark.parametrize("M,I,act,dtype", [(1, 128, "gelu", torch.bfloat16), (5, 256, "silu", torch.float32),
                                           (333, 512, "gelu", torch.float32), (1001, 384, "silu", torch.bfloat16)])
def test_backward(M, I, act, dtype, code, scale):
    bsmm = _bsmm()
    codes, scales = O.keep(gate_up(M, I, 5).float().numpy(), code, scale)
    g = torch.Generator().manual_seed(M)
    dh = torch.randn(M, I, generator=g).to(dtype)
    v = O.values(codes, scales, code)
    ref, href = O.gated_backward(dh.float().numpy(), v, act)
    d, h = bsmm.gated_act_backward(dh.cuda(), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), act=act,
                                   code=code, scale=scale, return_h=True)
    assert d.dtype == dtype and h.dtype == torch.bfloat16
    g64, u64 = v[:, :I].astype(np.float64), np.abs(v[:, I:].astype(np.float64))
    # act' is a sum of p and g p (1 - p), or of the CDF and g times the density: either may cancel
    mag = np.abs(dh.float().numpy()) * u64 * (1 + np.abs(g64) * np.exp(-np.minimum(np.abs(g64), 700) * 0.5))
    tol = np.concatenate([4 * REL * mag, REL * (np.abs(ref[:, I:]) + np.abs(dh.float().numpy()) * 1e-6)], 1)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23
    got = d.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - ref) <= tol + half * np.abs(ref) + 1e-37)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3], got[bad][:3], ref[bad][:3])
    hd = h.float().cpu().numpy()
    assert (np.abs(hd - href) <= (2.0 ** -8 + REL) * np.abs(href) + REL * 1e-6 * u64 + 1e-37).all()
    only, none = bsmm.gated_act_backward(dh.cuda(), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                                         act=act, code=code, scale=scale)
    assert none is None and torch.equal(only, d)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_against_differences(act):
    """Central differences of the float64 forward at the checkpoint's values."""
    bsmm = _bsmm()
    M, I, eps = 20, 256, 1e-5
    codes, scales = O.keep(torch.randn(M, 2 * I).numpy(), "int8", "f32")
    v = O.values(codes, scales, "int8").astype(np.float64)
    dh = torch.randn(M, I)
    d, _ = bsmm.gated_act_backward(dh.cuda(), torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), act=act)
    got = d.cpu().numpy().astype(np.float64)
    for half in (0, 1):
        step = np.zeros_like(v)
        step[:, half * I:(half + 1) * I] = eps
        diff = (O.gated(v + step, act) - O.gated(v - step, act)) / (2 * eps) * dh.numpy()
        # differences: eps^2 of the third derivative, 1e-16 / eps of rounding
        np.testing.assert_allclose(got[:, half * I:(half + 1) * I], diff, rtol=2e-5, atol=2e-5)


def test_bf16_gradient_is_the_rounded_f32_one():
    bsmm = _bsmm()
    M, I = 64, 256
    codes, scales = (torch.from_numpy(t).cuda() for t in O.keep(gate_up(M, I, 9).float().numpy(), "e4m3", "ue8m0"))
    dh = torch.randn(M, I, device="cuda").to(torch.bfloat16)
    kw = dict(code="e4m3", scale="ue8m0")
    a, _ = bsmm.gated_act_backward(dh, codes, scales, **kw)
    b, _ = bsmm.gated_act_backward(dh.float(), codes, scales, **kw)
    assert torch.equal(a, b.to(torch.bfloat16))


def test_empty():
    bsmm = _bsmm()
    z = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    h, hs, codes, scales = bsmm.gated_act(z)
    assert h.shape == (0, 128) and codes.shape == (0, 256) and scales.shape == (0, 2)
    d, _ = bsmm.gated_act_backward(z[:, :128], codes, scales)
    assert d.shape == (0, 256)


def _align(n, a=256):
    return (n + a - 1) // a * a


@pytest.mark.parametrize("M,N,K", [(32, 64, 128), (160, 96, 384), (2048, 160, 256)])
@pytest.mark.parametrize("code,scale", FORMATS)
@pytest.mark.parametrize("fp8", ["e4m3", "e5m2"])
def test_linear_backward_checkpoint(fp8, code, scale, M, N, K):
    """X^T as the call leaves it in the workspace equals the oracle's
    quantization of the checkpoint's values, bit for bit; dX and dW are those
    of the GEMMs on these operands, which an MXFP8 checkpoint's values, exact in
    bfloat16, reach through bsmm_linear_backward too."""
    bsmm = _bsmm()
    g = torch.Generator().manual_seed(M + N + K)
    dY = (torch.randn(M, N, generator=g) * 4).to(torch.bfloat16).cuda()
    W = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16).cuda()
    x = torch.randn(M, K, generator=g)
    x[:, 3] = 0
    codes, scales = O.keep(x.numpy(), code, scale)
    v = O.values(codes, scales, code)
    ws = torch.full((bsmm.linear_backward_workspace_size(M, N, K),), 0xA5, dtype=torch.uint8, device="cuda")
    dX, dW = bsmm.linear_backward_checkpoint(dY, W, torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                                             x_code=code, x_scale=scale, fp8=fp8, workspace=ws)
    assert bsmm.check_device_status()[0] == 0
    off = 0
    buf = ws.cpu().numpy()
    parts = []
    for rows, cols in ((M, N), (K, N), (N, M), (K, M)):
        n_atoms = bsmm.scale_atoms_size(1, rows, cols, fp8, "ue8m0")
        c = buf[off:off + rows * cols].reshape(rows, cols)
        off += _align(rows * cols)
        parts.append((c, buf[off:off + n_atoms]))
        off += _align(n_atoms)
    oc, osc = G.mx_quantize(v, "rows", fp8)
    np.testing.assert_array_equal(parts[3][0], oc)
    fmt = "mxfp8" if fp8 == "e4m3" else "mxfp8_e5m2"
    np.testing.assert_array_equal(decode_atoms(parts[3][1], 1, K, M, fmt)[0], osc)
    ops = [torch.from_numpy(np.ascontiguousarray(t)).cuda() for p in parts for t in p]
    rX, rW = bsmm.linear_backward_quantized(*ops, fp8=fp8, scales_are_atoms=True)
    assert torch.equal(dX, rX) and torch.equal(dW, rW)
    if scale == "ue8m0":
        bX, bW = bsmm.linear_backward(dY, W, torch.from_numpy(v).to(torch.bfloat16).cuda(), fp8)
        assert torch.equal(dX, bX) and torch.equal(dW, bW)
