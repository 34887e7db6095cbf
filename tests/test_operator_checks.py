"""What the adapter and checkpoint calls refuse, and their workspace queries,
without a GPU: the binding's checks of tensors (on CPU tensors, which the last
check refuses), and the library's checks before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_gb300 as bsmm
from oracle import adapters as A
from oracle import checkpoint as C
from oracle import quantize as Q


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return bsmm.lib()


CUDA = "must be a CUDA tensor"
fake = ctypes.c_void_p(4096)
odd = ctypes.c_void_p(4097)


def refused(fn, *args, match, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*args, **kw)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def ids(n):
    return z(n, dtype=torch.int32)


def test_adapters_binding():
    f = bsmm.adapters
    a, b = z(3, 4, 16), z(3, 8, 4)
    refused(f, z(5, 16, 1), a, b, ids(5), match="2-D")
    refused(f, z(5, 16), a[0], b, ids(5), match="\\(L, R, K\\)")
    refused(f, z(5, 16), a, z(3, 8, 5), ids(5), match="b must have shape \\(3, 8, 4\\)")
    refused(f, z(5, 16), a, z(2, 8, 4), ids(5), match="b must have shape")
    refused(f, z(5, 16), a.float(), b, ids(5), match="bfloat16")
    refused(f, z(5, 16), a, b, ids(4), match="ids must have shape \\(5,\\)")
    refused(f, z(5, 16), a, b, ids(5).long(), match="int32")
    refused(f, z(5, 16), a, b, ids(5), scaling=z(4, dtype=torch.float32), match="scaling must have shape")
    refused(f, z(5, 15), a, b, ids(5), match="x must have shape \\(5, 16\\)")
    refused(f, z(5, 16), a, b, ids(5), match=CUDA)
    refused(f, z(5, 16, dtype=torch.float32), a, b, ids(5), match="bfloat16")


def test_adapters_backward_binding():
    f = bsmm.adapters_backward
    a, b, u = z(3, 4, 32), z(3, 8, 4), z(5, 4, dtype=torch.float32)
    refused(f, z(5, 8, 1), z(5, 32), a, b, ids(5), u, match="2-D")
    refused(f, z(5, 9), z(5, 32), a, b, ids(5), u, match="dy must have shape \\(5, 8\\)")
    refused(f, z(5, 8), z(5, 32), a, b, ids(5), u, match=CUDA)


def test_gated_binding():
    f = bsmm.gated_act
    refused(f, z(4, 129), match="2 I")
    refused(f, z(4, 256, dtype=torch.float16), match="float32 or")
    refused(f, z(4, 256), codes=z(4, 255, dtype=torch.int8), match="codes must have shape")
    refused(f, z(4, 256), scales=z(4, 2), match="4-byte")
    refused(f, z(4, 256), h=z(4, 128), match="1-byte")
    refused(f, z(4, 256), match=CUDA)
    g = bsmm.gated_act_backward
    refused(g, z(4, 128), z(4, 128, dtype=torch.int8), z(4, 2, dtype=torch.float32), match="codes must have shape")
    refused(g, z(4, 128), z(4, 256, dtype=torch.int8), z(4, 3, dtype=torch.float32), match="scales must have shape")
    refused(g, z(4, 128), z(4, 256, dtype=torch.int8), z(4, 2, dtype=torch.float32), match=CUDA)


def test_linear_binding():
    f = bsmm.linear_backward_checkpoint
    c = z(64, 128, dtype=torch.uint8)
    refused(f, z(64, 32), z(32, 128), c, z(64, 3, dtype=torch.uint8), match="x_scales must have shape \\(64, 4\\)")
    refused(f, z(64, 32), z(32, 128), c[:, :64], z(64, 4, dtype=torch.uint8), match="x_codes must have shape")
    refused(f, z(64, 32), z(32, 128), c, z(64, 4, dtype=torch.uint8), match=CUDA)


def adapters_args(**kw):
    d = dict(T=4, K=64, N=32, R=8, L=2, x=fake, ld_x=64, A=fake, B=fake, ids=fake, s=None, y=fake, ld_y=32, out=fake,
             ld_out=32, yt=bsmm.BF16, u=fake, ws=None, wb=0, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), bsmm.ERR_INVALID_ARG), (dict(K=0), bsmm.ERR_SHAPE), (dict(R=0), bsmm.ERR_SHAPE),
    (dict(L=0), bsmm.ERR_SHAPE), (dict(R=129), bsmm.ERR_UNSUPPORTED), (dict(yt=bsmm.E4M3), bsmm.ERR_INVALID_ARG),
    (dict(x=None), bsmm.ERR_INVALID_ARG), (dict(u=None), bsmm.ERR_INVALID_ARG), (dict(ld_x=63), bsmm.ERR_SHAPE),
    (dict(ld_y=31), bsmm.ERR_SHAPE), (dict(ld_y=40), bsmm.ERR_SHAPE), (dict(x=odd), bsmm.ERR_ALIGNMENT),
    (dict(ids=ctypes.c_void_p(4098)), bsmm.ERR_ALIGNMENT), (dict(T=8192), bsmm.ERR_WORKSPACE),
    (dict(T=8192, ws=fake, wb=100), bsmm.ERR_WORKSPACE), (dict(T=0, x=None, out=None), bsmm.OK)])
def test_adapters_library(lib, change, status):
    assert lib.bsmm_adapters(*adapters_args(**change)) == status


def backward_args(**kw):
    d = dict(T=4, K=64, N=32, R=8, L=2, dy=fake, ld_dy=32, x=fake, ld_x=64, xt=bsmm.BF16, xs=None, A=fake, B=fake,
             ids=fake, s=None, u=fake, base=None, ld_dx=64, dx=fake, dA=fake, dB=fake, gt=bsmm.F32, ws=fake,
             wb=1 << 20, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), bsmm.ERR_INVALID_ARG), (dict(R=200), bsmm.ERR_UNSUPPORTED), (dict(gt=bsmm.INT8), bsmm.ERR_INVALID_ARG),
    (dict(xt=bsmm.INT8), bsmm.ERR_INVALID_ARG), (dict(xt=bsmm.E4M3), bsmm.ERR_INVALID_ARG),
    (dict(xs=fake), bsmm.ERR_INVALID_ARG), (dict(K=40, ld_x=40, ld_dx=40, xt=bsmm.E4M3, xs=fake), bsmm.ERR_SHAPE),
    (dict(ld_x=96, xt=bsmm.E4M3, xs=fake), bsmm.ERR_SHAPE), (dict(ld_dy=31), bsmm.ERR_SHAPE),
    (dict(dA=None), bsmm.ERR_INVALID_ARG), (dict(ws=None), bsmm.ERR_WORKSPACE), (dict(wb=127), bsmm.ERR_WORKSPACE), (dict(L=1025), bsmm.ERR_UNSUPPORTED),
    (dict(ws=ctypes.c_void_p(4100)), bsmm.ERR_WORKSPACE), (dict(dy=odd), bsmm.ERR_ALIGNMENT)])
def test_adapters_backward_library(lib, change, status):
    assert lib.bsmm_adapters_backward(*backward_args(**change)) == status


def gated_args(**kw):
    d = dict(x=fake, xt=bsmm.BF16, M=4, I=128, ld=256, act=bsmm.SILU, ht=bsmm.E4M3, h=fake, hs=fake, atoms=0,
             ct=bsmm.INT8, st=bsmm.SCALE_F32, codes=fake, scales=fake, stream=None)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("change,status", [
    (dict(xt=bsmm.E4M3), bsmm.ERR_INVALID_ARG), (dict(act=2), bsmm.ERR_INVALID_ARG), (dict(ht=bsmm.INT8), bsmm.ERR_INVALID_ARG),
    (dict(M=-1), bsmm.ERR_INVALID_ARG), (dict(st=bsmm.SCALE_UE8M0), bsmm.ERR_UNSUPPORTED),
    (dict(ct=bsmm.E2M1), bsmm.ERR_UNSUPPORTED), (dict(st=bsmm.SCALE_UE4M3, ct=bsmm.E4M3), bsmm.ERR_UNSUPPORTED),
    (dict(I=96, ld=192), bsmm.ERR_SHAPE), (dict(I=40, ld=80, codes=None), bsmm.ERR_SHAPE), (dict(ld=255), bsmm.ERR_SHAPE),
    (dict(ld=260), bsmm.ERR_ALIGNMENT), (dict(h=odd), bsmm.ERR_ALIGNMENT), (dict(hs=None), bsmm.ERR_INVALID_ARG),
    (dict(scales=None), bsmm.ERR_INVALID_ARG), (dict(scales=ctypes.c_void_p(4098)), bsmm.ERR_ALIGNMENT),
    (dict(M=0, x=None, h=None), bsmm.OK)])
def test_gated_library(lib, change, status):
    assert lib.bsmm_gated_act(*gated_args(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dt=bsmm.E4M3), bsmm.ERR_INVALID_ARG), (dict(act=-1), bsmm.ERR_INVALID_ARG), (dict(I=-1), bsmm.ERR_INVALID_ARG),
    (dict(st=bsmm.SCALE_UE8M0), bsmm.ERR_UNSUPPORTED), (dict(I=96), bsmm.ERR_SHAPE), (dict(dh=None), bsmm.ERR_INVALID_ARG),
    (dict(h=odd), bsmm.ERR_ALIGNMENT), (dict(codes=odd), bsmm.ERR_ALIGNMENT), (dict(M=0, dh=None), bsmm.OK)])
def test_gated_backward_library(lib, change, status):
    d = dict(dh=fake, dt=bsmm.BF16, M=4, I=128, act=bsmm.GELU, codes=fake, ct=bsmm.INT8, scales=fake, st=bsmm.SCALE_F32,
             d=fake, h=None, stream=None)
    d.update(change)
    assert lib.bsmm_gated_act_backward(*d.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(ft=bsmm.INT8), bsmm.ERR_INVALID_ARG), (dict(xt=bsmm.INT8), bsmm.ERR_UNSUPPORTED), (dict(M=33), bsmm.ERR_SHAPE),
    (dict(xt=bsmm.INT8, st=bsmm.SCALE_F32, K=96), bsmm.ERR_SHAPE), (dict(x=None), bsmm.ERR_INVALID_ARG),
    (dict(x=odd), bsmm.ERR_ALIGNMENT), (dict(wb=64), bsmm.ERR_WORKSPACE), (dict(N=0, dY=None), bsmm.OK)])
def test_linear_library(lib, change, status):
    d = dict(dY=fake, W=fake, x=fake, xt=bsmm.E4M3, xs=fake, st=bsmm.SCALE_UE8M0, M=64, N=64, K=128, ft=bsmm.E5M2,
             dX=fake, dW=fake, ws=fake, wb=1 << 24, stream=None)
    d.update(change)
    assert lib.bsmm_linear_backward_checkpoint(*d.values()) == status


def test_workspace_query(lib):
    assert bsmm.adapters_workspace_size(64, 16, 64) == 0  # few tokens are not sorted
    assert bsmm.adapters_workspace_size(8192, 16, 4) >= 8192 * 4
    assert bsmm.adapters_backward_workspace_size(0, 8, 4) == 0
    assert bsmm.adapters_backward_workspace_size(100, 8, 4) >= 100 * 8 * 4 + 100 * 4


def test_oracle_adapters_are_a_dense_product_per_token():
    rng = np.random.default_rng(3)
    x, a, b = rng.normal(size=(6, 5)), rng.normal(size=(2, 3, 5)), rng.normal(size=(2, 4, 3))
    ids, s, dy = np.array([0, 1, -1, 1, 2, 0]), np.array([0.5, 2.0]), rng.normal(size=(6, 4))
    out, u = A.forward(x, a, b, ids, scaling=s)
    for t, k in enumerate(ids):
        full = s[k] * (b[k] @ a[k]) if 0 <= k < 2 else np.zeros((4, 5))
        np.testing.assert_allclose(out[t], full @ x[t], atol=1e-12)
    dx, da, db, _ = A.backward(dy, x, a, b, ids, u, scaling=s)
    for name, grad in (("x", dx), ("a", da), ("b", db)):  # the forward is linear in each
        v = {"x": x, "a": a, "b": b}
        step = rng.normal(size=v[name].shape)
        moved = {**v, name: v[name] + step}
        diff = ((A.forward(**moved, ids=ids, scaling=s)[0] - out) * dy).sum()
        np.testing.assert_allclose(diff, (grad * step).sum(), rtol=1e-10)


def test_oracle_checkpoint_agrees_with_the_quantizer():
    x = np.random.default_rng(4).normal(size=(8, 256)).astype(np.float32)
    x[2] = 0
    for code in ("e4m3", "e5m2"):
        kept, ref = C.keep(x, code, "ue8m0"), Q.quantize(x, (1, 32), code, "ue8m0")
        np.testing.assert_array_equal(kept[0], ref[0])
        np.testing.assert_array_equal(kept[1], ref[1])
    for code in ("int8", "e4m3", "e5m2"):  # binary32 scales: at most one ulp apart
        kept, ref = C.keep(x, code, "f32"), Q.quantize(x, (1, 128), code, "f32")
        assert (np.abs(kept[1] - ref[1]) <= np.spacing(ref[1])).all()
        assert (np.abs(C.values(*kept, code) - x) <= np.abs(x).max() / (127 if code == "int8" else 4)).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_oracle_gated_slope_against_differences(act):
    g = np.linspace(-6, 6, 97)
    f, df = C.act(g, act)
    eps = 1e-6
    np.testing.assert_allclose(df, (C.act(g + eps, act)[0] - C.act(g - eps, act)[0]) / (2 * eps), atol=1e-8)
