"""The launches that work on many tokens, each of which may start before the
one ahead of it ends: what follows a call on its stream finds all of the call's
outputs, whatever the tokens' adapters."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


@pytest.mark.parametrize("K,N", [(67, 45), (1031, 45), (64, 72)])
@pytest.mark.parametrize("some", [False, True])
def test_tokens_without_adapters(K, N, some):
    """No token has an adapter, or only the last one of 2100: u is zero and out
    is y by the time that the next work of the stream reads them, in calls
    that follow each other on one workspace."""
    bsmm = _bsmm()
    T, R, L = 2100, 16, 3
    g = torch.Generator(device="cuda").manual_seed(K)
    x, a, b, y, dy, base = (torch.randn(*s, device="cuda", generator=g).bfloat16()
                            for s in ((T, K), (L, R, K), (L, N, R), (T, N), (T, N), (T, K)))
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    if some:
        ids[-1] = 1
    ws = torch.empty(bsmm.adapters_workspace_size(T, R, L), dtype=torch.uint8, device="cuda")
    back = torch.empty(bsmm.adapters_backward_workspace_size(T, R, L), dtype=torch.uint8, device="cuda")
    out, u, dx = torch.empty_like(y), torch.empty((T, R), device="cuda"), torch.empty_like(base)
    seen = []
    for _ in range(20):
        u.fill_(float("nan"))
        out.fill_(float("nan"))
        bsmm.adapters(x, a, b, ids, y=y, out=out, u=u, workspace=ws)
        seen.append((u.clone(), out.clone()))
        _, da, db = bsmm.adapters_backward(dy, x, a, b, ids, u, dx_base=base, dx=dx, workspace=back)
        seen[-1] += (dx.clone(), da, db)
    for su, so, sx, da, db in seen:
        assert not su[:-1].any() and torch.equal(so[:-1], y[:-1]) and torch.equal(sx[:-1], base[:-1])
        assert bool(su[-1].all()) == some and bool(da[1].any()) == some and bool(db[1].any()) == some
        assert not da[::2].any() and not db[::2].any()
    assert bsmm.check_device_status()[0] == 0


@pytest.mark.parametrize("K", [32, 96, 160, 416, 256])
@pytest.mark.parametrize("R,grad", [(8, torch.float32), (16, torch.bfloat16), (64, torch.float32)])
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_checkpoint_like_its_values(K, R, grad, order):
    """Codes and scales, whose rows may end inside a 4-byte word, give the bits
    that their values, exact in bfloat16, give: a scale read before it is there
    would not."""
    bsmm = _bsmm()
    T, N, L = 4200, 136, 3
    g = torch.Generator(device="cuda").manual_seed(K + R)
    wide = torch.exp2(torch.randint(-20, 20, (T, K // 32), device="cuda", generator=g).float()).repeat_interleave(32, 1)
    codes, scales = bsmm.quantize(torch.randn(T, K, device="cuda", generator=g) * wide, (1, 32), "e4m3", "ue8m0")
    values = codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127).repeat_interleave(32, 1)
    x = values.bfloat16()
    assert torch.equal(x.float(), values)
    a, b, dy = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((L, R, K), (L, N, R), (T, N)))
    u = torch.randn(T, R, device="cuda", generator=g)
    ids = torch.randint(-1, L, (T,), device="cuda", dtype=torch.int32, generator=g)
    if order == "runs":
        ids = ids.sort().values
    ref = bsmm.adapters_backward(dy, x, a, b, ids, u, grad_dtype=grad)
    for _ in range(5):
        got = bsmm.adapters_backward(dy, codes, a, b, ids, u, x_scales=scales, grad_dtype=grad)
        for p, q in zip(ref, got):
            assert torch.equal(p, q)
    assert bsmm.check_device_status()[0] == 0


@pytest.mark.parametrize("T,K,N", [(8, 64, 40), (8, 63, 41), (2100, 64, 72), (16500, 67, 45)])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_gradients_of_adapters_without_tokens(T, K, N, grad):
    """Zero, also where the scaling is no finite number; the last tokens alone
    use adapter 1."""
    bsmm = _bsmm()
    R, L = 16, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    x, a, b, dy = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((T, K), (L, R, K), (L, N, R), (T, N)))
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[-5:] = 1
    u = torch.randn(T, R, device="cuda", generator=g)
    scaling = torch.tensor([float("nan"), 0.5, float("inf"), -float("inf")], device="cuda")
    _, da, db = bsmm.adapters_backward(dy, x, a, b, ids, u, scaling=scaling, grad_dtype=grad)
    for t in (da, db):
        assert not t[[0, 2, 3]].any() and bool(torch.isfinite(t[1].float()).all()) and bool(t[1].any())
    scaling[1] = float("nan")
    _, da, db = bsmm.adapters_backward(dy, x, a, b, ids, u, scaling=scaling, grad_dtype=grad)
    assert bool(da[1].isnan().all()) and bool(db[1].isnan().all()) and not da[::2].any() and not db[::2].any()
