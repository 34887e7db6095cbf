"""u and d reach the second product of bsmm_adapters and its backward as the
binary32 numbers that they are, whatever the outputs' type.

Rank 0 holds 1 + 2^-9 + 2^-20, rank 1 holds 1 + 2^-9, and the output is their
difference: 2^-20 exactly, in every order of the additions (all partial sums
have at most 21 significant bits).  A u cut to 16 bits loses it whole."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _pair(rows, at):
    """[rows, 2] or its transpose: rank 0 takes the first three columns, rank 1 two of them."""
    w = torch.zeros(2, rows)
    w[0, :3] = 1
    w[1, :2] = 1
    return w.t() if at else w


# few tokens as they come, tiles with TMA, tiles of rows that are not 16-byte aligned
@pytest.mark.parametrize("T,K,N", [(1, 64, 96), (5, 37, 45), (40, 512, 264), (2112, 128, 136), (2112, 67, 45)])
@pytest.mark.parametrize("R", [2, 16, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_second_product_keeps_every_bit(T, K, N, R, dtype):
    bsmm = _bsmm()
    bits = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -20])
    a, b = torch.zeros(1, R, K), torch.zeros(1, N, R)
    a[0, :2] = _pair(K, False)
    b[0, :, 0], b[0, :, 1] = 1, -1
    x = torch.zeros(T, K)
    x[:, :3] = bits
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    cu = lambda t: t.bfloat16().cuda()  # noqa: E731
    out, u = bsmm.adapters(cu(x), cu(a), cu(b), ids, out_dtype=dtype)
    assert bool((u[:, 0] == bits.double().sum()).all()) and bool((u[:, 1] == 1 + 2.0 ** -9).all())
    assert bool((out == 2.0 ** -20).all())
    # the same with a base that the product cancels: -(1 + 2^-7), exact in both types
    a[0, 1] = 0
    base = torch.full((T, N), -1.0, dtype=dtype, device="cuda")
    out, _ = bsmm.adapters(cu(x), cu(a), cu(b), ids, y=base)
    want = torch.tensor(2.0 ** -9 + 2.0 ** -20).to(dtype)
    assert bool((out == want.cuda()).all())

    # backward: d = B^T dy, dx = A^T d
    b, a = torch.zeros(1, N, R), torch.zeros(1, R, K)
    b[0, :, :2] = _pair(N, True)
    a[0, 0], a[0, 1] = 1, -1
    dy = torch.zeros(T, N)
    dy[:, :3] = bits
    dx, _, _ = bsmm.adapters_backward(cu(dy), cu(x), cu(a), cu(b), ids, torch.zeros(T, R, device="cuda"))
    assert bool((dx == 2.0 ** -20).all())
