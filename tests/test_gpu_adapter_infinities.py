"""Infinities in weights, tokens and sums give what the formulas give in 64
bits: the same places are infinite, with the same signs, and NaN.

The inputs are random normal numbers, none of them zero, so that the formulas
give NaN only where infinities cancel.  The finite results are held to 2^-6 of
their root mean square: other tests hold them closer."""

import numpy as np
import pytest
import torch

from oracle import adapters as O
from oracle import checkpoint as C

pytestmark = pytest.mark.gpu
INF = float("inf")


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def same(got, ref, what):
    got = _f64(got)
    ref = ref.astype(np.float32)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    at = np.isinf(ref)
    np.testing.assert_array_equal(np.isinf(got), at, err_msg=what)
    np.testing.assert_array_equal(np.sign(got[at]), np.sign(ref[at]), err_msg=what)
    fine = np.isfinite(ref)
    rms = np.sqrt(np.mean(ref[fine].astype(np.float64) ** 2)) if fine.any() else 0.0
    assert (np.abs(got[fine] - ref[fine]) <= 2.0 ** -6 * (rms + np.abs(ref[fine]))).all(), what


SHAPES = [(6, 64, 96), (41, 264, 136), (41, 71, 45), (2112, 64, 72), (2112, 67, 45)]


def make(T, K, N, R, L=5):
    g = torch.Generator().manual_seed(T + K + N + R)

    def rnd(*s):
        t = torch.randn(*s, generator=g).to(torch.bfloat16)
        t[t == 0] = 0.5
        return t

    ids = (torch.arange(T) % (L + 1) - 1).to(torch.int32)
    return rnd(T, K), rnd(L, R, K), rnd(L, N, R), rnd(T, N), ids


def first(ids, k):
    return int(torch.nonzero(ids == k)[0, 0])


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("R", [4, 16, 33, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward(T, K, N, R, dtype):
    x, a, b, y, ids = make(T, K, N, R)
    y = y.to(dtype)
    b[1, 7, 1] = INF            # a weight of the second product: u there is finite
    b[1, 9] = -INF
    a[2, 0, 5] = -INF           # one infinite u a token
    x[first(ids, 3), 4] = INF   # all of a token's u
    scaling = torch.tensor([0.5, -1.0, 2.0, 0.25, 1.0])
    with np.errstate(invalid="ignore"):
        ref, uref = O.forward(_f64(x), _f64(a), _f64(b), _f64(ids), _f64(y), _f64(scaling))
    out, u = _bsmm().adapters(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), y=y.cuda(), scaling=scaling.cuda())
    same(u, uref, "u")
    same(out, ref, "out")


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("R", [4, 16, 64, 128])
@pytest.mark.parametrize("x_code", [None, "e5m2"])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_backward(T, K, N, R, x_code, grad):
    if x_code and K % 32:
        K = 96
    bsmm = _bsmm()
    x, a, b, dy, ids = make(T, K, N, R)
    dy[first(ids, 1), 13] = INF
    a[2, 1, 5] = -INF
    b[4, 3, 2] = INF
    g = torch.Generator().manual_seed(3)
    u = torch.randn(T, R, generator=g) + 3.0 * torch.sign(torch.randn(T, R, generator=g))
    u[first(ids, 0), 1] = -INF
    sick = first(ids, 3)
    kw = {}
    if x_code:
        codes, scales = bsmm.quantize(x.cuda(), (1, 32), x_code, "ue8m0")
        codes[sick, 6] = 0x7C  # infinity
        codes[(codes & 0x7F) == 0] = 1
        x64 = C.values(codes.cpu().numpy(), scales.cpu().numpy(), x_code).astype(np.float64)
        xg, kw = codes, dict(x_scales=scales, x_code=x_code)
    else:
        x[sick, 6] = -INF
        x64, xg = _f64(x), x.cuda()
    with np.errstate(invalid="ignore"):
        rdx, rda, rdb, _ = O.backward(_f64(dy), x64, _f64(a), _f64(b), _f64(ids), _f64(u))
    dx, da, db = bsmm.adapters_backward(dy.cuda(), xg, a.cuda(), b.cuda(), ids.cuda(), u.cuda(), grad_dtype=grad, **kw)
    same(dx, rdx, "dx")
    same(da, rda, "dA")
    same(db, rdb, "dB")


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_numbers_beside_the_largest(T, K, N, dtype):
    """u = (2 - 2^-8) 2^127, finite, which bfloat16 rounds to infinity."""
    x, a, b = torch.zeros(T, K), torch.zeros(1, 1, K), torch.full((1, N, 1), 2.0 ** -100)
    x[:, 0], x[:, 1] = (2 - 2.0 ** -7) * 2.0 ** 127, 2.0 ** 119
    a[0, 0, :2] = 1
    cu = lambda t: t.bfloat16().cuda()  # noqa: E731
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    out, u = _bsmm().adapters(cu(x), cu(a), cu(b), ids, out_dtype=dtype)
    want = (2 - 2.0 ** -8) * 2.0 ** 27
    assert bool((u == want * 2.0 ** 100).all())
    assert bool((out == torch.tensor(want).to(dtype).cuda()).all())
