"""The softmax over all experts, entry by entry, on logits that lie far apart.

U = 2^-24.  An entry's exponential e^x, x = l - m: x is rounded, |x| U of the entry;
the function is off by 4 U, two roundings and 0.22 |x| U: (1.22 |x| + 6) U, and by
2^-126 where it counts as zero.  In the sum of all, |x| counts by its mean under
the softmax, at most ln E <= 7: 15 U, and 32 + 5 additions: 52 U.  A weight: its own
exponential (expf, 4 U) and the sum's errors, a quotient: (|x| + 57) U.

A gradient of an expert that is not chosen, p mean: p as above, (1.22 |x| + 6 + 52) U,
a quotient and a product: (1.22 |x| + 60) U of p |mean|; the mean of k products
through five levels of sums is off by 6 U of mag = sum |w dw|.  A chosen one adds w
dw, two roundings of mag and of itself.  A bfloat16 result adds 2^-8 of itself."""

import numpy as np
import pytest
import torch

from oracle import experts as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _f64(t):
    return t.detach().double().cpu().numpy()


def logits_of(T, E, span, dtype):
    """Rows spread evenly over `span`, and rows with a crowd at either end."""
    g = torch.Generator().manual_seed(T + E + span)
    l = torch.rand(T, E, generator=g) * span
    l[1::3] = torch.where(torch.rand(T, E, generator=g) < 0.9, l / 8, l)[1::3]
    l[2::3] = torch.where(torch.rand(T, E, generator=g) < 0.9, span - l / 8, l)[2::3]
    return (l - span / 3).to(dtype).cuda()


CASES = [(40, 16, 4, 8), (70, 96, 5, 20), (64, 1024, 32, 50), (300, 256, 8, 80), (33, 1000, 3, 100), (200, 30, 3, 86),
         (5, 512, 6, 200)]


@pytest.mark.parametrize("T,E,k,span", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights(T, E, k, span, dtype):
    l = logits_of(T, E, span, dtype)
    w, ids, *_ = _bsmm().route(l, k, renormalize=False)
    ref, ref_ids = O.route(_f64(l), k, False)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    x = _f64(l).max(1, keepdims=True) - np.take_along_axis(_f64(l), ref_ids.astype(np.int64), 1)
    assert (np.abs(_f64(w) - ref) <= (x + 57) * U * ref + 2.0 ** -148).all()


@pytest.mark.parametrize("T,E,k,span", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1.0, 1e6])
def test_gradient_entry_by_entry(T, E, k, span, dtype, size):
    bsmm = _bsmm()
    l = logits_of(T, E, span, dtype)
    w, ids, *_ = bsmm.route(l, k, renormalize=False)
    dw = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(E)) * size
    got = _f64(bsmm.route_backward(dw, l, ids, w, renormalize=False))
    w64, dw64, l64, at = _f64(w), _f64(dw), _f64(l), ids.cpu().numpy().astype(np.int64)
    ref = O.route_backward(dw64, l64, ids.cpu().numpy(), w64, False)
    mag = np.abs(w64 * dw64).sum(1, keepdims=True)
    mean = np.abs((w64 * dw64).sum(1, keepdims=True))
    x = l64.max(1, keepdims=True) - l64
    p = np.exp(-x) / np.exp(-x).sum(1, keepdims=True)
    tol = (1.22 * x + 60) * U * p * mean + 6 * U * p * mag + 2.0 ** -126 * (mean + 1)
    chosen = np.zeros(l64.shape, bool)
    np.put_along_axis(chosen, at, True, 1)
    tol = tol + np.where(chosen, 2 * U * (mag + np.abs(ref)), 0)
    if dtype is torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
