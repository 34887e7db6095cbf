"""What the calls of a mixture of experts and the AdamW step refuse, and their
workspace queries, without a GPU: the binding's checks (on CPU tensors, which
the last check refuses) and the library's checks before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

import block_scaled_precision_gemm_gb300 as bsmm
from oracle import adamw as A
from oracle import experts as X


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return bsmm.lib()


CUDA = "CUDA tensor"
fake = ctypes.c_void_p(4096)
odd = ctypes.c_void_p(4097)


def refused(fn, *args, match, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        fn(*args, **kw)


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return z(*shape, dtype=torch.int32)


def u8(*shape):
    return z(*shape, dtype=torch.uint8)


def f32(*shape):
    return z(*shape, dtype=torch.float32)


def test_route_binding(lib):
    refused(bsmm.route, z(4, 8, 1), 2, match="2-D")
    refused(bsmm.route, z(4, 8, dtype=torch.float16), 2, match="float32 or")
    refused(bsmm.route, z(4, 8), 2, match=CUDA)
    f = bsmm.route_backward
    refused(f, f32(4, 2), z(4, 8, 1), i32(4, 2), f32(4, 2), match="2-D")
    refused(f, f32(4, 2), z(4, 8), i32(4, 2), f32(4, 2), match=CUDA)


def test_expert_gemm_binding(lib):
    f = bsmm.expert_gemm
    x, xs, w, a, o = u8(10, 64), u8(10, 2), u8(3, 32, 64), u8(3 * 2 * 1 * 512), i32(4)
    refused(f, x, xs, w[0], a, o, match="\\[E, N, K\\]")
    refused(f, x.float(), xs, w, a, o, match="1-byte")
    refused(f, x, xs[:, :1], w, a, o, match="x_scales must have shape \\(10, 2\\)")
    refused(f, x, xs, u8(3, 32, 96), a, o, match="w must have shape")
    refused(f, x, xs, w, a[:-1], o, match=r"bytes, \d+ needed")
    refused(f, x, xs, w, a, i32(3), match="offsets must have shape \\(4,\\)")
    refused(f, x, xs, w, a, o.long(), match="int32")
    refused(f, x, xs, w, a, o, rows=i32(2, 2), match="1-D")
    refused(f, x, xs, w, a, o, rows=i32(5), y=z(10, 32), match="y must have shape \\(5, 32\\)")
    refused(f, x, xs, w, a, o, y=f32(10, 32), match="bfloat16")
    refused(f, x, xs, w, a, o, match=CUDA)


def test_expert_backward_binding(lib):
    f = bsmm.expert_backward
    dY, W, x, o = z(10, 32), z(3, 32, 64), z(10, 64), i32(4)
    refused(f, dY, W[0], x, o, match="\\[E, N, K\\]")
    refused(f, dY.float(), W, x, o, match="bfloat16")
    refused(f, dY[:9], W, x, o, match="dY must have shape \\(10, 32\\)")
    refused(f, dY, W, z(10, 32), o, match="X must have shape")
    refused(f, dY, W, x, o, rows=i32(9), match="dY must have shape \\(9, 32\\)")
    refused(f, dY, W, x, o, dW=z(3, 64, 32), match="dW must have shape")
    refused(f, dY, W, x, o, match=CUDA)


def test_combine_binding(lib):
    f, g = bsmm.expert_combine, bsmm.expert_combine_backward
    y, s = z(8, 16), i32(4, 2)
    refused(f, y.float(), s, match="bfloat16")
    refused(f, y, s.long(), match="int32")
    refused(f, y, s[0], match="\\[T, k\\]")
    refused(f, y, s, f32(4, 3), match="weights must have shape \\(4, 2\\)")
    refused(f, y, s, out_dtype=torch.float16, match="float32 or")
    refused(f, y, s, out=z(4, 15), match="out must have shape")
    refused(f, y, s, match=CUDA)
    refused(g, z(4, 15), y, s, match="d_out must have shape")
    refused(g, z(4, 16), y, s, f32(4, 2), dy=z(7, 16), match="dy must have shape")
    refused(g, z(4, 16), y, s, match=CUDA)


def test_adamw_binding(lib):
    f = bsmm.adamw
    p, kw = [f32(5), f32(200)], dict(step=1, lr=0.1)
    refused(f, p, [f32(5)], p, p, match="grads holds 1 tensors|CUDA", **kw)
    refused(f, [1.0], p, p, p, match="Tensors", **kw)
    refused(f, [f32(5), z(200)], p, p, p, match="one type", **kw)
    refused(f, [f32(5).half(), f32(200).half()], p, p, p, match="float32 or", **kw)
    refused(f, p, p, p, p, m_scales=[f32(1), f32(2)], match="go together", **kw)
    refused(f, p, p, p, p, match=CUDA, **kw)


def status(fn, base, change):
    d = dict(base)
    d.update(change)
    return fn(*d.values())


ROUTE = dict(T=300, E=8, k=2, l=fake, lt=bsmm.F32, ld=8, r=1, ids=fake, w=fake, off=fake, rows=fake, slots=fake, ws=fake,
             wb=1 << 20, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), bsmm.ERR_INVALID_ARG), (dict(lt=bsmm.E4M3), bsmm.ERR_INVALID_ARG), (dict(k=0), bsmm.ERR_SHAPE),
    (dict(k=9), bsmm.ERR_SHAPE), (dict(E=1025, ld=1025), bsmm.ERR_UNSUPPORTED), (dict(E=64, ld=64, k=33), bsmm.ERR_UNSUPPORTED),
    (dict(T=1 << 31), bsmm.ERR_SHAPE), (dict(ld=7), bsmm.ERR_SHAPE), (dict(l=None), bsmm.ERR_INVALID_ARG),
    (dict(off=None), bsmm.ERR_INVALID_ARG), (dict(l=odd), bsmm.ERR_ALIGNMENT), (dict(ids=odd), bsmm.ERR_ALIGNMENT),
    (dict(ws=None), bsmm.ERR_WORKSPACE), (dict(wb=64), bsmm.ERR_WORKSPACE), (dict(ws=ctypes.c_void_p(4100)), bsmm.ERR_WORKSPACE)])
def test_route_library(lib, change, want):
    assert status(lib.bsmm_route, ROUTE, change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=0), bsmm.ERR_SHAPE), (dict(l=None, r=0), bsmm.ERR_INVALID_ARG), (dict(dl=None), bsmm.ERR_INVALID_ARG),
    (dict(dl=odd), bsmm.ERR_ALIGNMENT), (dict(T=0, dl=None), bsmm.OK)])
def test_route_backward_library(lib, change, want):
    assert status(lib.bsmm_route_backward, dict(T=4, E=8, k=2, l=fake, lt=bsmm.BF16, ld=8, r=1, dw=fake, ids=fake, w=fake,
                                                dl=fake, stream=None), change) == want


@pytest.mark.parametrize("change,want", [
    (dict(S=-1), bsmm.ERR_INVALID_ARG), (dict(xt=bsmm.INT8), bsmm.ERR_INVALID_ARG), (dict(wt=bsmm.BF16), bsmm.ERR_INVALID_ARG),
    (dict(N=40), bsmm.ERR_SHAPE), (dict(K=48), bsmm.ERR_SHAPE), (dict(K=0), bsmm.ERR_SHAPE), (dict(E=0), bsmm.ERR_SHAPE),
    (dict(E=1025), bsmm.ERR_UNSUPPORTED), (dict(X=9), bsmm.ERR_SHAPE), (dict(X=0, rows=fake), bsmm.ERR_SHAPE),
    (dict(E=1024, N=1 << 20, K=1 << 20), bsmm.ERR_SHAPE), (dict(S=(1 << 30) + 1, X=(1 << 30) + 1), bsmm.ERR_SHAPE),
    (dict(x=None), bsmm.ERR_INVALID_ARG), (dict(off=None), bsmm.ERR_INVALID_ARG), (dict(x=ctypes.c_void_p(4104)), bsmm.ERR_ALIGNMENT),
    (dict(rows=odd), bsmm.ERR_ALIGNMENT), (dict(S=4000, rows=fake), bsmm.ERR_WORKSPACE),
    (dict(S=4000, rows=fake, ws=fake, wb=64), bsmm.ERR_WORKSPACE), (dict(S=0, x=None, y=None), bsmm.OK)])
def test_expert_gemm_library(lib, change, want):
    assert status(lib.bsmm_expert_gemm, dict(S=10, X=10, E=4, N=64, K=128, x=fake, xt=bsmm.E4M3, xs=fake, w=fake, wt=bsmm.E4M3,
                                             a=fake, off=fake, rows=None, y=fake, ws=None, wb=0, stream=None), change) == want


@pytest.mark.parametrize("change,want", [
    (dict(ft=bsmm.INT8), bsmm.ERR_INVALID_ARG), (dict(N=40), bsmm.ERR_SHAPE), (dict(X=9), bsmm.ERR_SHAPE),
    (dict(dW=None), bsmm.ERR_INVALID_ARG), (dict(dX=None), bsmm.ERR_INVALID_ARG), (dict(W=odd), bsmm.ERR_ALIGNMENT),
    (dict(dW=odd), bsmm.ERR_ALIGNMENT), (dict(ws=None), bsmm.ERR_WORKSPACE), (dict(wb=100), bsmm.ERR_WORKSPACE),
    (dict(ws=ctypes.c_void_p(4112)), bsmm.ERR_WORKSPACE)])
def test_expert_backward_library(lib, change, want):
    assert status(lib.bsmm_expert_backward, dict(S=10, X=10, E=4, N=64, K=128, dY=fake, W=fake, x=fake, off=fake, rows=None,
                                                 ft=bsmm.E5M2, dX=fake, dW=fake, ws=fake, wb=1 << 26, stream=None), change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=0), bsmm.ERR_SHAPE), (dict(k=33), bsmm.ERR_UNSUPPORTED), (dict(N=0), bsmm.ERR_SHAPE), (dict(T=-1), bsmm.ERR_INVALID_ARG),
    (dict(t=bsmm.E4M3), bsmm.ERR_INVALID_ARG), (dict(y=None), bsmm.ERR_INVALID_ARG), (dict(o=odd), bsmm.ERR_ALIGNMENT),
    (dict(T=0, o=None), bsmm.OK)])
def test_combine_library(lib, change, want):
    assert status(lib.bsmm_expert_combine, dict(T=4, S=8, k=2, N=16, y=fake, s=fake, w=fake, o=fake, t=bsmm.F32, stream=None),
                  change) == want


@pytest.mark.parametrize("change,want", [
    (dict(k=0), bsmm.ERR_SHAPE), (dict(d=None), bsmm.ERR_INVALID_ARG), (dict(w=None), bsmm.ERR_INVALID_ARG),
    (dict(dy=None), bsmm.ERR_INVALID_ARG), (dict(dy=odd), bsmm.ERR_ALIGNMENT), (dict(T=0, d=None), bsmm.OK)])
def test_combine_backward_library(lib, change, want):
    assert status(lib.bsmm_expert_combine_backward, dict(T=4, S=8, k=2, N=16, d=fake, t=bsmm.F32, y=fake, s=fake, w=fake, dy=fake,
                                                         dw=fake, stream=None), change) == want


def pointers(*v):
    return (ctypes.c_uint64 * len(v))(*v)


@pytest.mark.parametrize("change,want", [
    (dict(count=-1), bsmm.ERR_INVALID_ARG), (dict(pt=bsmm.E4M3), bsmm.ERR_INVALID_ARG), (dict(st=bsmm.BF16), bsmm.ERR_INVALID_ARG),
    (dict(lr=-1.0), bsmm.ERR_INVALID_ARG), (dict(lr=float("nan")), bsmm.ERR_INVALID_ARG), (dict(b1=1.0), bsmm.ERR_INVALID_ARG),
    (dict(b2=-0.1), bsmm.ERR_INVALID_ARG), (dict(step=0), bsmm.ERR_INVALID_ARG), (dict(p=None), bsmm.ERR_INVALID_ARG),
    (dict(n=(ctypes.c_int64 * 2)(5, -1)), bsmm.ERR_INVALID_ARG), (dict(p=pointers(4096, 0)), bsmm.ERR_INVALID_ARG),
    (dict(g=pointers(4096, 4098)), bsmm.ERR_ALIGNMENT), (dict(st=bsmm.E4M3), bsmm.ERR_INVALID_ARG),
    (dict(st=bsmm.E4M3, ms=pointers(4096, 4096), vs=pointers(4096, 4098)), bsmm.ERR_ALIGNMENT),
    (dict(c=pointers(0, 4097)), bsmm.ERR_ALIGNMENT), (dict(hyper=odd), bsmm.ERR_ALIGNMENT), (dict(count=0, p=None), bsmm.OK)])
def test_adamw_library(lib, change, want):
    two = pointers(4096, 4096)
    base = dict(count=2, n=(ctypes.c_int64 * 2)(5, 6), p=two, pt=bsmm.F32, g=two, gt=bsmm.F32, m=two, v=two, st=bsmm.F32, ms=None,
                vs=None, c=None, lr=0.1, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, s=1.0, hyper=None, stream=None)
    assert status(lib.bsmm_adamw, base, change) == want


def test_workspace_queries(lib):
    assert bsmm.route_workspace_size(4, 64) == 0  # few tokens take one launch
    assert bsmm.route_workspace_size(100000, 64) > 0 and bsmm.route_workspace_size(0, 64) == 0
    assert bsmm.expert_gemm_workspace_size(8, 4, 64) == 0 and bsmm.expert_gemm_workspace_size(4000, 4, 64, False) == 0
    assert bsmm.expert_gemm_workspace_size(4000, 4, 64) >= 4000 * 66
    assert bsmm.expert_backward_workspace_size(0, 4, 64, 64) == 0
    assert bsmm.expert_backward_workspace_size(100, 4, 64, 64) >= 100 * 64 + 4 * 64 * 64 + 2 * 64 * 100


def test_oracle_layout_and_sums():
    rng = np.random.default_rng(1)
    w, ids = X.route(rng.normal(size=(9, 5)), 2, True)
    offsets, rows, slots = X.layout(ids, 5)
    assert (rows[slots] == np.arange(9)[:, None]).all() and offsets[-1] == 18
    for e in range(5):
        assert sorted(slots[ids == e]) == list(range(offsets[e], offsets[e + 1]))
    x = rng.normal(size=(9, 4))
    np.testing.assert_allclose(X.combine(x[rows], slots, w)[0], x, atol=1e-12)  # weights sum to 1
    y = rng.normal(size=(18, 4))
    d = rng.normal(size=(9, 4))
    dy, dw, _ = X.combine_backward(d, y, slots, w)
    step = rng.normal(size=y.shape)
    np.testing.assert_allclose(((X.combine(y + step, slots, w)[0] - X.combine(y, slots, w)[0]) * d).sum(), (dy * step).sum())
    np.testing.assert_allclose((X.combine(y, slots, w)[0] * d).sum(), (w * dw).sum())


def test_oracle_adamw_forms_agree():
    rng = np.random.default_rng(2)
    p, g, m, v = rng.normal(size=300), rng.normal(size=300), rng.normal(size=300), rng.random(300)
    a = A.step(p, g, m, v, 5, 1e-2, (0.9, 0.99), 1e-8, 0.1)
    b = A.step32(p, g, m, v, 5, 1e-2, (0.9, 0.99), 1e-8, 0.1)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-4, atol=1e-5)
    s = A.scales(m)
    assert (np.abs(A.values(A.codes(m, s), s) - m) <= np.abs(m) * 2.0 ** -4 + s.max() * 2.0 ** -10).all()
