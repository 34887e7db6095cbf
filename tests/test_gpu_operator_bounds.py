"""The adapters and the checkpoint operators write nothing outside their
outputs and workspaces: each is the interior of a larger device buffer whose
margins hold a sentinel, and the shapes end inside tiles, blocks and pieces.
Padded rows of an output at a wider pitch keep what they held."""

import pytest
import torch

pytestmark = pytest.mark.gpu
MARGIN = 1 << 16
SENTINEL = 0xA5


class Guarded:
    """A tensor of `shape` and `dtype` inside a sentinel-filled buffer."""

    def __init__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        self.nbytes = n * torch.empty((), dtype=dtype).element_size()
        self.buf = torch.full((2 * MARGIN + self.nbytes,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.t = self.buf[MARGIN:MARGIN + self.nbytes].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        assert bool((self.buf[:MARGIN] == SENTINEL).all()) and bool((self.buf[MARGIN + self.nbytes:] == SENTINEL).all())


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


@pytest.mark.parametrize("T,K,N,R,L,runs", [(1, 72, 40, 5, 2, False), (37, 130, 201, 12, 5, False),
                                            (700, 328, 264, 24, 3, False), (700, 323, 261, 24, 3, False),
                                            (1300, 264, 392, 64, 2, True), (300, 136, 200, 128, 2, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adapters(T, K, N, R, L, runs, dtype):
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(T + K)

    def t(*s):
        return torch.randn(*s, device="cuda", generator=g).bfloat16()

    x, a, b, y, dy = t(T, K), t(L, R, K), t(L, N, R), t(T, N).to(dtype), t(T, N)
    ids = torch.randint(-1, L, (T,), device="cuda", dtype=torch.int32, generator=g)
    if runs:
        ids = ids.sort().values
    wide = N + 24  # a pitch whose padding must stay
    out, u = Guarded((T, wide), dtype), Guarded((T, R), torch.float32)
    before = out.t.view(torch.uint8)[:, N * out.t.element_size():].clone()
    ws = Guarded((max(bsmm.adapters_workspace_size(T, R, L), 256),), torch.uint8)
    bsmm.adapters(x, a, b, ids, y=y, out=out.t[:, :N], u=u.t, workspace=ws.t)
    for m in (out, u, ws):
        m.check()
    assert torch.equal(out.t.view(torch.uint8)[:, N * out.t.element_size():], before)
    assert bool(torch.isfinite(out.t[:, :N].float()).all()) and bool(torch.isfinite(u.t).all())

    dx, da, db = Guarded((T, K), torch.bfloat16), Guarded((L, R, K), dtype), Guarded((L, N, R), dtype)
    ws = Guarded((bsmm.adapters_backward_workspace_size(T, R, L),), torch.uint8)
    bsmm.adapters_backward(dy, x, a, b, ids, u.t, grad_dtype=dtype, dx=dx.t, da=da.t, db=db.t, workspace=ws.t)
    for m in (dx, da, db, ws):
        m.check()
        if m is not ws:
            assert bool(torch.isfinite(m.t.float()).all())
    assert bsmm.check_device_status()[0] == 0


@pytest.mark.parametrize("M,I", [(1, 128), (37, 384), (131, 1152)])
@pytest.mark.parametrize("code,scale", [("int8", "f32"), ("e4m3", "ue8m0"), ("e5m2", "f32")])
def test_gated_act(M, I, code, scale):
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(M + I)
    gate_up = torch.randn(M, 2 * I, device="cuda", generator=g).bfloat16()
    dh = torch.randn(M, I, device="cuda", generator=g).bfloat16()
    block, sdt = (128, torch.float32) if scale == "f32" else (32, torch.uint8)
    h, hs = Guarded((M, I), torch.uint8), Guarded((M, I // 32), torch.uint8)
    codes, scales = Guarded((M, 2 * I), torch.uint8), Guarded((M, 2 * I // block), sdt)
    bsmm.gated_act(gate_up, code=code, scale=scale, h=h.t, h_scales=hs.t, codes=codes.t, scales=scales.t)
    atoms = Guarded((bsmm.scale_atoms_size(1, M, I, bsmm.E4M3, bsmm.SCALE_UE8M0),), torch.uint8)
    bsmm.gated_act(gate_up, code=None, h=h.t, h_scales=atoms.t, h_scales_are_atoms=True)
    d, hb = Guarded((M, 2 * I), torch.bfloat16), Guarded((M, I), torch.bfloat16)
    bsmm.gated_act_backward(dh, codes.t, scales.t, code=code, scale=scale, d_gate_up=d.t, h=hb.t)
    for m in (h, hs, codes, scales, atoms, d, hb):
        m.check()
    assert bool(torch.isfinite(d.t.float()).all()) and bool(torch.isfinite(hb.t.float()).all())


@pytest.mark.parametrize("M,N,K", [(32, 64, 128), (288, 160, 384), (1056, 416, 128)])
def test_linear_backward_checkpoint(M, N, K):
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(M)
    dY, W, X = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((M, N), (N, K), (M, K)))
    for block, code, scale in (((1, 128), "int8", "f32"), ((1, 32), "e4m3", "ue8m0")):
        c, s = bsmm.quantize(X, block, code, scale)
        dX, dW = Guarded((M, K), torch.bfloat16), Guarded((N, K), torch.bfloat16)
        ws = Guarded((bsmm.linear_backward_workspace_size(M, N, K),), torch.uint8)
        bsmm.linear_backward_checkpoint(dY, W, c, s, x_code=code, x_scale=scale, dX=dX.t, dW=dW.t, workspace=ws.t)
        for m in (dX, dW, ws):
            m.check()
        assert bool(torch.isfinite(dX.t.float()).all()) and bool(torch.isfinite(dW.t.float()).all())
    assert bsmm.check_device_status()[0] == 0
