"""Gradients of long sums: all tokens of one adapter, so many that every CTA
ends several rounds of its accumulators (a round is at most 60 blocks of 64
tokens for ranks up to 16 and 24 beyond, and a cluster of at most 8 CTAs shares
the blocks); and contractions over many columns.

The 2-norm of a binary32 gradient's error is held to 1e-6 of its norm.  The
tensor cores cut off what does not fit: an addition loses 2^-24 of the running
sum on average, and in a round of 48 additions that sum grows as the root of
their number, so a round's drift is 48 * 2^-24 * 2/3 = 1.9e-6 of its own sum; the
sums of the rounds, sets and CTAs (at least 10 of them) are independent and so
is their drift's sign, which leaves 1.9e-6 / sqrt(10) = 6e-7.  Additions without
rounds, 100 and more to an accumulator, come out above 1e-6."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


CASES = [  # T, K, N, R, L: aligned, then odd widths
    (62000, 64, 72, 16, 1), (62000, 96, 64, 8, 1), (25200, 64, 72, 24, 1), (25200, 32, 72, 32, 1), (25200, 64, 40, 64, 1),
    (25200, 96, 64, 128, 1), (65600, 1024, 1000, 16, 8),
    (62000, 64, 71, 16, 1), (25200, 64, 71, 24, 1), (25200, 32, 45, 64, 1), (25200, 64, 33, 128, 1),
    (65600, 992, 1001, 16, 8), (65600, 992, 1001, 64, 8),
]


@pytest.mark.parametrize("T,K,N,R,L", CASES)
@pytest.mark.parametrize("x_code", [None, "e4m3"])
def test_long_sums_of_one_adapter(T, K, N, R, L, x_code):
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(T + K + N + R)

    def rnd(*s, k=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * k).bfloat16()

    x, dy, a, b = rnd(T, K), rnd(T, N), rnd(L, R, K, k=K ** -0.5), rnd(L, N, R, k=R ** -0.5)
    u = torch.randn(T, R, device="cuda", generator=g)
    ids = torch.full((T,), L // 2, dtype=torch.int32, device="cuda")
    kw, x64 = {}, x.double()
    if x_code:
        xq, xs = bsmm.quantize(x, (1, 32), x_code, "ue8m0")
        x64 = (xq.view(torch.float8_e4m3fn).float() * torch.exp2(xs.float() - 127).repeat_interleave(32, 1)).double()
        x, kw = xq, dict(x_scales=xs, x_code=x_code)
    scaling = torch.linspace(0.5, 1.5, L, device="cuda")
    _, da, db = bsmm.adapters_backward(dy, x, a, b, ids, u, scaling=scaling, **kw)
    k, s = L // 2, float(scaling[L // 2])
    wa = s * (dy.double() @ b[k].double()).t() @ x64
    wb = s * dy.double().t() @ u.double()
    assert _rel(da[k], wa) < 1e-6 and _rel(db[k], wb) < 1e-6
    rest = [i for i in range(L) if i != k]
    assert not da[rest].any() and not db[rest].any()
    # and in bfloat16: half an ulp, 2^-9 at most
    _, ha, hb = bsmm.adapters_backward(dy, x, a, b, ids, u, scaling=scaling, grad_dtype=torch.bfloat16, **kw)
    assert _rel(ha[k], wa) < 2.0 ** -9 and _rel(hb[k], wb) < 2.0 ** -9
    assert bsmm.check_device_status()[0] == 0


@pytest.mark.parametrize("T,K,N", [(262144, 512, 512), (262144, 511, 513)])
def test_lower_terms_of_high_ranks(T, K, N):
    """Ranks above 32 sum the coefficients' lower terms, 2^-8 of them, in an
    accumulator of their own, which has to end its rounds too: here a CTA takes
    1024 blocks or more of the one adapter in use, 8200 additions without rounds."""
    bsmm = _bsmm()
    R, L = 128, 8
    g = torch.Generator(device="cuda").manual_seed(N)

    def rnd(*s, k=1.0):
        return (torch.randn(*s, device="cuda", generator=g) * k).bfloat16()

    x, dy, a, b = rnd(T, K), rnd(T, N), rnd(L, R, K, k=K ** -0.5), rnd(L, N, R, k=R ** -0.5)
    u = torch.randn(T, R, device="cuda", generator=g)
    ids = torch.full((T,), 2, dtype=torch.int32, device="cuda")
    _, da, db = bsmm.adapters_backward(dy, x, a, b, ids, u)
    assert _rel(da[2], (dy.double() @ b[2].double()).t() @ x.double()) < 1e-6
    assert _rel(db[2], dy.double().t() @ u.double()) < 1e-6


@pytest.mark.parametrize("T,K", [(20000, 8192), (20000, 8191), (40000, 16384), (24000, 6000)])
@pytest.mark.parametrize("R", [16, 24, 64, 128])
@pytest.mark.parametrize("order", ["runs", "mixed"])
def test_long_contractions(T, K, R, order):
    """u of so many tokens that a tile has one CTA, which ends its rounds over all
    of K: at most 48 additions to an accumulator, as for the gradients.  Consecutive
    tokens, whose rows come by TMA alone, and scattered ones."""
    bsmm = _bsmm()
    N, L = 64, 2
    g = torch.Generator(device="cuda").manual_seed(T + K + R)
    x, b = (torch.randn(*s, device="cuda", generator=g).bfloat16() for s in ((T, K), (L, N, R)))
    a = (torch.randn(L, R, K, device="cuda", generator=g) * K ** -0.5).bfloat16()
    ids = (torch.arange(T, device="cuda") * L // T if order == "runs" else torch.arange(T, device="cuda") % L).int()
    out, u = bsmm.adapters(x, a, b, ids, out_dtype=torch.float32)
    want = torch.empty(T, R, dtype=torch.float64, device="cuda")
    for k in range(L):
        want[ids == k] = x[ids == k].double() @ a[k].double().t()
    assert _rel(u, want) < 1e-6
    # d, seen through dA (x of FP8 adds its own part: 3e-7)
    dy, db = x, a.transpose(1, 2).contiguous()  # N = K here
    small, s = bsmm.quantize(torch.randn(T, 64, device="cuda", generator=g), (1, 32), "e4m3", "ue8m0")
    x64 = (small.view(torch.float8_e4m3fn).float() * torch.exp2(s.float() - 127).repeat_interleave(32, 1)).double()
    _, da, _ = bsmm.adapters_backward(dy, small, b[:, :, :].transpose(1, 2).contiguous(), db, ids, u, x_scales=s)
    for k in range(L):
        assert _rel(da[k], want[ids == k].t() @ x64[ids == k]) < 1e-6
    assert bsmm.check_device_status()[0] == 0
