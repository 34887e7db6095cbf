"""bsmm_route, bsmm_route_backward and the sums of the experts' results against
their float64 forms.

Choices and layouts are equal, ties to the lowest index.  Weights: the binary32
difference to the largest logit is off by 2^-24 of itself, which the
exponential turns into that much relative error; expf adds 2 ulp (2^-22), the
quotient half of one, and a sum of positive terms in binary32 over at most 32
terms a lane and five levels at most 37 2^-24: (range + 48) 2^-24 of the weight
in all.  A product's sum of n terms in binary32 is off by at most (n + 1) 2^-24
of the sum of magnitudes; a bfloat16 result adds 2^-8 of the value."""

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


def _i(t):
    return t.cpu().numpy()


def logits_of(T, E, dtype, seed=0, ties=False):
    g = torch.Generator().manual_seed(1000 * seed + 31 * T + E)
    l = torch.randn(T, E, generator=g) * 2
    if ties:
        l = torch.round(l * 2) / 2
        l[l == 0] = -0.0  # -0 and 0 tie
        l[::2, ::3] = l[::2, ::3].clamp(min=0.0)
    return l.to(dtype).cuda()


def check_route(l, k, renormalize, **kw):
    bsmm = _bsmm()
    weights, ids, offsets, rows, slots = bsmm.route(l, k, renormalize=renormalize, **kw)
    ref, ref_ids = O.route(_f64(l), k, renormalize)
    np.testing.assert_array_equal(_i(ids), ref_ids)
    for got, want in zip((offsets, rows, slots), O.layout(ref_ids, l.shape[1])):
        np.testing.assert_array_equal(_i(got), want)
    finite = np.where(np.isfinite(_f64(l)), _f64(l), 0)
    span = (finite.max(1) - finite.min(1))[:, None]
    assert (np.abs(_f64(weights) - ref) <= (span + 48) * U * ref).all()
    return weights, ids, offsets, rows, slots


ROUTES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (16, 64, 4), (7, 33, 8), (128, 64, 8), (129, 64, 8), (127, 256, 6),
          (300, 33, 7), (1000, 128, 2), (2000, 256, 8), (130, 1000, 32), (64, 1024, 32), (513, 1024, 4), (4097, 7, 2),
          (260, 512, 1), (65, 256, 8), (64, 256, 16), (66, 40, 17)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(T, E, k, dtype, renormalize):
    check_route(logits_of(T, E, dtype), k, renormalize)


@pytest.mark.parametrize("T,E,k", [(20011, 64, 4), (9000, 300, 10), (30007, 6, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(T, E, k, dtype):
    """Several tokens a warp, the last blocks and runs partial."""
    check_route(logits_of(T, E, dtype, ties=dtype is torch.bfloat16), k, False)


@pytest.mark.parametrize("T", [9, 777])
@pytest.mark.parametrize("E,k", [(8, 3), (40, 8), (256, 16)])
def test_ties_go_to_the_lowest_index(T, E, k):
    check_route(logits_of(T, E, torch.bfloat16, ties=True), k, True)
    check_route(torch.zeros(T, E, device="cuda"), k, False)


@pytest.mark.parametrize("T", [12, 900])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_experts_and_tokens(T, renormalize):
    l = logits_of(T, 40, torch.float32)
    l[:, 7] = -float("inf")
    l[1] = -float("inf")          # nothing left
    l[2, 3:] = -float("inf")      # fewer than k left
    l[3] = float("nan")
    l[4, ::2] = float("nan")
    l[5] = torch.finfo(torch.float32).min  # the lowest number is chosen all the same
    w, ids, offsets, rows, slots = check_route(l, 5, renormalize)
    assert (_i(ids)[[1, 3]] == -1).all() and (_i(slots)[[1, 3]] == -1).all()
    used = int(offsets[-1])
    assert used < T * 5 and (_i(rows)[used:] == -1).all()


def test_infinite_logits_choose_and_weigh_as_the_formula():
    l = logits_of(4, 16, torch.float32)
    l[2, 9] = float("inf")
    w, ids, *_ = _bsmm().route(l, 3)
    assert int(ids[2, 0]) == 9 and bool(torch.isnan(w[2, 0]))
    assert bool(torch.isfinite(w[[0, 1, 3]]).all())


def test_no_tokens():
    w, ids, offsets, rows, slots = _bsmm().route(torch.empty(0, 12, device="cuda"), 3)
    assert w.shape == (0, 3) and rows.shape == (0,) and _i(offsets).tolist() == [0] * 13
    d = _bsmm().route_backward(w, torch.empty(0, 12, device="cuda"), ids, w)
    assert d.shape == (0, 12)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [20, 700])
def test_rows_at_a_pitch(T, dtype):
    wide = logits_of(T, 71, dtype)
    check_route(wide[:, 3:67], 6, False)
    l = wide[:, 3:67]
    w, ids, *_ = _bsmm().route(l, 6, renormalize=False)
    dw = torch.randn(T, 6, device="cuda")
    for r in (True, False):
        assert torch.equal(_bsmm().route_backward(dw, l, ids, w, renormalize=r),
                           _bsmm().route_backward(dw, l.contiguous(), ids, w, renormalize=r))


@pytest.mark.parametrize("T,E,k", ROUTES[:14:2] + [(1003, 96, 5)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward(T, E, k, dtype, renormalize):
    bsmm = _bsmm()
    l = logits_of(T, E, dtype)
    if E > 4:
        l[0, 1] = -float("inf")
        l[-1, 0] = float("nan")
    w, ids, *_ = bsmm.route(l, k, renormalize=renormalize)
    dw = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    got = _f64(bsmm.route_backward(dw, l, ids, w, renormalize=renormalize))
    ref = O.route_backward(_f64(dw), _f64(l), _i(ids), _f64(w), renormalize)
    # mean: k + 1 roundings of |w dw|; p: as the weights'; three products after it
    mag = (np.abs(_f64(w)) * np.abs(_f64(dw))).sum(1)[:, None]
    finite = np.where(np.isfinite(_f64(l)), _f64(l), 0)
    span = (finite.max(1) - finite.min(1))[:, None]
    tol = (k + span + 60) * U * (mag + np.abs(ref)) + (2.0 ** -8 * np.abs(ref) if dtype is torch.bfloat16 else 0)
    assert (np.abs(got - ref) <= tol + 1e-38).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_against_differences(renormalize):
    """The weights' directional derivative, float64 differences of the definition."""
    bsmm = _bsmm()
    l = logits_of(6, 10, torch.float32)
    w, ids, *_ = bsmm.route(l, 3, renormalize=renormalize)
    dw = torch.randn(6, 3, device="cuda")
    got = _f64(bsmm.route_backward(dw, l, ids, w, renormalize=renormalize))
    step = np.random.default_rng(0).normal(size=(6, 10))
    h = 1e-5  # smaller than half the gaps between logits: the choice stays
    hi, lo = (O.route(_f64(l) + s * h * step, 3, renormalize) for s in (1, -1))
    assert (hi[1] == _i(ids)).all() and (lo[1] == _i(ids)).all()
    want = ((hi[0] - lo[0]) / (2 * h) * _f64(dw)).sum()
    assert abs((got * step).sum() - want) <= 1e-5 * np.abs(got * step).sum() + 1e-8


def test_route_backward_of_ids_by_hand():
    """Ids outside the experts have no part; one given twice adds up."""
    l = logits_of(3, 6, torch.float32)
    ids = torch.tensor([[2, 2], [-1, 5], [6, 0]], dtype=torch.int32, device="cuda")
    w, dw = torch.rand(3, 2, device="cuda"), torch.randn(3, 2, device="cuda")
    for r in (True, False):
        got = _f64(_bsmm().route_backward(dw, l, ids, w, renormalize=r))
        ref = O.route_backward(_f64(dw), _f64(l), _i(ids), _f64(w), r)
        np.testing.assert_allclose(got, ref, rtol=1e-5, atol=1e-6)


def pairs(T, S, k, seed=0, dropped=True):
    g = torch.Generator().manual_seed(seed + T + S)
    slots = torch.randperm(S, generator=g)[:T * k].view(T, k).to(torch.int32)
    if dropped:
        slots[0, 0] = -1
        slots[-1, -1] = S
        if T > 2:
            slots[1] = -1
    return slots.cuda()


COMBINES = [(1, 1, 8), (1, 4, 4096), (16, 4, 513), (33, 2, 1024), (5, 8, 2056), (300, 3, 96), (7, 32, 264), (64, 1, 1),
            (2, 17, 40)]


# many tokens (smaller blocks), and rows of more columns than a block takes
COMBINES += [(700, 4, 4104), (640, 2, 513), (1300, 1, 72), (2, 3, 9000), (650, 9, 40)]


@pytest.mark.parametrize("T,k,N", COMBINES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, N, dtype, weighted):
    bsmm = _bsmm()
    S = T * k + 5
    g = torch.Generator("cuda").manual_seed(T * N)
    y = torch.randn(S, N, device="cuda", generator=g).bfloat16()
    slots = pairs(T, S, k, dropped=T * k > 2)
    y[int(set(range(S)).difference(_i(slots).flatten().tolist()).pop())] = float("nan")  # a slot of no token
    w = torch.randn(T, k, device="cuda", generator=g) if weighted else None
    out = bsmm.expert_combine(y, slots, w, out_dtype=dtype)
    ref, mag = O.combine(np.nan_to_num(_f64(y)), _i(slots), None if w is None else _f64(w))
    tol = (k + 1) * U * mag + (2.0 ** -8 * np.abs(ref) if dtype is torch.bfloat16 else 0)
    assert (np.abs(_f64(out) - ref) <= tol).all()

    d = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    dy = torch.full_like(y, 7.0)
    got, dw = bsmm.expert_combine_backward(d, y, slots, w, dy=dy)
    ref, ref_w, mag = O.combine_backward(_f64(d), np.nan_to_num(_f64(y)), _i(slots), None if w is None else _f64(w))
    left = np.isnan(ref)
    assert (_f64(got)[left] == 7.0).all()
    assert (np.abs(_f64(got) - ref)[~left] <= (2.0 ** -8 + U) * np.abs(ref)[~left]).all()
    if weighted:
        assert (np.abs(_f64(dw) - ref_w) <= (N + 1) * U * mag).all()
    else:
        assert dw is None


def test_combine_unaligned_rows():
    """A view that starts between two 16-byte pieces gives the same bits."""
    bsmm = _bsmm()
    flat = torch.randn(9 * 64 + 1, device="cuda").bfloat16()
    y, slots = flat[1:].view(9, 64), pairs(4, 9, 2)
    w, d = torch.rand(4, 2, device="cuda"), torch.randn(4, 64, device="cuda")
    assert torch.equal(bsmm.expert_combine(y, slots, w), bsmm.expert_combine(y.clone(), slots, w))
    a, b = (bsmm.expert_combine_backward(d, t, slots, w, dy=torch.zeros(9, 64, device="cuda").bfloat16())
            for t in (y, y.clone()))
    assert torch.equal(a[0], b[0])
    torch.testing.assert_close(a[1], b[1], rtol=1e-5, atol=1e-5)


def test_combine_past_32_bits():
    """Rows whose first element lies beyond 2^31."""
    bsmm = _bsmm()
    N, S = 65536, 32800
    y = torch.zeros(S, N, device="cuda", dtype=torch.bfloat16)
    y[S - 1] = torch.arange(N, device="cuda") % 128
    slots = torch.tensor([[S - 1, 0], [1, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, 1.0], [1.0, 1.0]], device="cuda")
    out = bsmm.expert_combine(y, slots, w)
    assert torch.equal(out[0].float(), 2 * (torch.arange(N, device="cuda") % 128).float()) and not out[1].any()
    d = torch.ones(2, N, device="cuda").bfloat16()
    dy, dw = bsmm.expert_combine_backward(d, y, slots, w, dy=torch.zeros_like(y))
    assert float(dw[0, 0]) == float((torch.arange(N) % 128).sum())
    assert bool((dy[S - 1] == 2).all()) and not dy[S - 2].any()
