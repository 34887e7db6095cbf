"""bsmm_expert_gemm and bsmm_expert_backward against their float64 forms.

Products of MXFP8 values are exact in binary32; a sum of n of them is off by at
most n 2^-23 of the sum of magnitudes, even if every addition truncates, and the
bfloat16 result by half a step, 2^-8 of the value at most.  The backward's
operands are the quantizer's, bit for bit, so the same bound holds for it."""

import numpy as np
import pytest
import torch

from oracle import experts as O

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _f64(t):
    return t.detach().double().cpu().numpy()


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def check(got, ref, mag, n, left=None):
    """left: the value that rows of no expert keep."""
    got = _f64(got)
    untouched = np.isnan(ref)
    if untouched.any():
        assert (got[untouched] == left).all()
    tol = n * STEP * mag + 2.0 ** -8 * np.abs(ref) + 1e-38
    bad = ~(np.abs(got - ref) <= tol) & ~untouched
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def make(counts, N, K, rows=None, x_type="e4m3", w_type="e4m3", seed=0):
    """x, W in MXFP8 with scales spread over 2^-6 .. 2^6; rows: None or the number of x's rows."""
    bsmm = _bsmm()
    E, S = len(counts), int(sum(counts))
    g = torch.Generator("cuda").manual_seed(seed + 17 * S + N + K)
    X = max(S, 1) if rows is None else rows

    def rnd(r):
        spread = torch.exp2(torch.randint(-6, 7, (r, K // 32, 1), device="cuda", generator=g).float())
        return (torch.randn(r, K // 32, 32, device="cuda", generator=g) * spread).view(r, K)

    xv, wv = rnd(X), rnd(E * N)
    x, xs = bsmm.quantize(xv, (1, 32), x_type, "ue8m0")
    w, ws = bsmm.quantize(wv, (1, 32), w_type, "ue8m0")
    _, atoms = bsmm.quantize_atoms(wv, w_type, batches=E)
    d = {"x": x, "x_scales": xs, "w": w.view(E, N, K), "w_atoms": atoms, "x_type": x_type, "w_type": w_type,
         "rows": None if rows is None else torch.randint(0, X, (S,), device="cuda", generator=g, dtype=torch.int32)}
    d["xv"] = O.mx_values(x.cpu().numpy(), xs.cpu().numpy(), x_type)
    d["wv"] = O.mx_values(w.cpu().numpy(), ws.cpu().numpy(), w_type).reshape(E, N, K)
    return d


def run(d, offsets, **kw):
    return _bsmm().expert_gemm(d["x"], d["x_scales"], d["w"], d["w_atoms"], offsets, rows=d["rows"], x_type=d["x_type"],
                               w_type=d["w_type"], **kw)


GEMMS = [  # counts, N, K, rows of x
    ([1], 32, 32, None), ([1], 256, 128, 5), ([0, 3], 64, 96, None), ([5, 0, 0, 2], 160, 64, 3),
    ([255], 256, 256, None), ([256], 288, 128, 40), ([257, 1], 512, 128, None), ([33, 64, 0, 31, 32], 96, 544, 70),
    ([16] * 16, 256, 512, 20), ([1] * 40, 128, 1024, 8), ([700, 3, 130], 544, 640, None), ([700, 3, 130], 544, 640, 901),
    ([129, 128, 127, 385], 1024, 1536, 300), ([0, 0, 0], 64, 64, None), ([90, 1, 0, 600, 17, 64], 320, 2048, 64)]


@pytest.mark.parametrize("counts,N,K,rows", GEMMS)
def test_gemm(counts, N, K, rows):
    d = make(counts, N, K, rows)
    S = sum(counts)
    off = offsets_of(counts)
    y = run(d, off, y=torch.full((S if rows is not None else max(S, 1), N), 3.0, device="cuda").bfloat16())
    r = None if d["rows"] is None else d["rows"].cpu().numpy()
    check(y, *O.gemm(d["xv"], d["wv"], off.cpu().numpy(), r, y.shape[0]), K, left=3.0)
    assert _bsmm().check_device_status()[0] == 0


@pytest.mark.parametrize("x_type,w_type", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("rows", [None, 50])
def test_gemm_types(x_type, w_type, rows):
    counts = [40, 7, 300]
    d = make(counts, 160, 384, rows, x_type, w_type)
    off = offsets_of(counts)
    y = run(d, off)
    r = None if rows is None else d["rows"].cpu().numpy()
    check(y, *O.gemm(d["xv"], d["wv"], off.cpu().numpy(), r, sum(counts)), 384)


def test_gemm_more_tiles_than_clusters():
    """Every tile width, several tiles a cluster, both ways to the rows."""
    counts = [32 * i - (i % 5) for i in range(1, 13)]
    for rows in (None, 999):
        d = make(counts, 1312, 256, rows)
        off = offsets_of(counts)
        r = None if rows is None else d["rows"].cpu().numpy()
        check(run(d, off), *O.gemm(d["xv"], d["wv"], off.cpu().numpy(), r, sum(counts)), 256)


def test_gemm_many_experts():
    counts = [(i * 7) % 5 for i in range(1024)]
    d = make(counts, 32, 64, 100)
    off = offsets_of(counts)
    check(run(d, off), *O.gemm(d["xv"], d["wv"], off.cpu().numpy(), d["rows"].cpu().numpy(), sum(counts)), 64)


@pytest.mark.parametrize("rows", [None, 64])
def test_slots_of_no_expert_stay(rows):
    """Offsets that begin late and end early, and values outside the slots."""
    counts = [20, 30, 50]
    d = make(counts, 96, 128, rows)
    S = 100
    for off in ([7, 20, 20, 81], [-5, 40, 60, 400], [100, 100, 100, 100], [0, 0, 0, 0], [3, 4, 4, 4]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = run(d, o, y=torch.full((S, 96), -2.0, device="cuda").bfloat16())
        r = None if rows is None else d["rows"].cpu().numpy()
        check(y, *O.gemm(d["xv"], d["wv"], off, r, S), 128, left=-2.0)


def test_rows_of_no_token_reach_only_their_slot():
    counts = [30, 40]
    d = make(counts, 64, 128, 16)
    off = offsets_of(counts)
    want = run(d, off)
    at = [3, 29, 30, 69]
    d["rows"][at] = torch.tensor([-1, 16, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    keep = [i for i in range(70) if i not in at]
    assert torch.equal(run(d, off)[keep], want[keep])


@pytest.mark.parametrize("rows", [None, 40])
def test_nan_reaches_its_row_and_feature_only(rows):
    counts = [20, 50]
    d = make(counts, 96, 256, rows)
    off = offsets_of(counts)
    want = run(d, off)
    d["x_scales"][5, 3] = 255  # a NaN scale
    d["w"][1, 70, 9] = 0x7F    # a NaN code
    bad = _f64(run(d, off))
    hit = np.zeros_like(bad, bool)
    hit[20:, 70] = True
    hit[[5] if rows is None else np.flatnonzero(d["rows"].cpu().numpy() == 5)] = True
    assert (np.isnan(bad) == hit).all()
    assert (bad[~hit] == _f64(want)[~hit]).all()


@pytest.mark.parametrize("counts", [[10, 0, 3, 40], [100, 0, 260, 90]])
@pytest.mark.parametrize("K", [96, 640])
def test_rows_by_number_or_copied(counts, K):
    """Few rows an expert are fetched by number, many are copied ahead: both give
    the bits of rows that lie in the slots' order."""
    d = make(counts, 288, K, 77)
    off = offsets_of(counts)
    at = d["rows"].long()
    e = dict(d, x=d["x"][at], x_scales=d["x_scales"][at], rows=None)
    assert torch.equal(run(d, off), run(e, off))


@pytest.mark.parametrize("off", [[0, 70, 20, 90, 60], [90, 0, 90, 0, 90], [-2 ** 31, 2 ** 31 - 1, -1, 50, 2]])
def test_offsets_that_fall_stay_inside(off):
    """Offsets that are none: unspecified sums, in their own arrays."""
    bsmm = _bsmm()
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    d = make([30, 20, 20, 20], 96, 128, 40)

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        flat = torch.full((n + 8192,), 77, device="cuda").to(dtype)
        return flat, flat[4096:4096 + n].view(shape)

    fy, y = guarded((90, 96), torch.bfloat16)
    run(d, o, y=y)
    dY, W, X, r = backward_inputs([30, 20, 20, 20], 96, 128, 40)
    fx, dX = guarded((90, 128), torch.bfloat16)
    fw, dW = guarded((4, 96, 128), torch.bfloat16)
    need = bsmm.expert_backward_workspace_size(90, 4, 96, 128)
    fs, ws = guarded((need,), torch.uint8)
    bsmm.expert_backward(dY, W, X, o, rows=r, dX=dX, dW=dW, workspace=ws)
    torch.cuda.synchronize()
    for f in (fy, fx, fw, fs):
        assert bool((f[:4096] == f[0]).all()) and bool((f[-4096:] == f[0]).all())
    assert bsmm.check_device_status()[0] == 0


def test_gemm_past_32_bits():
    """An output of more than 2^32 bytes: its last rows."""
    bsmm = _bsmm()
    S, N, K = 66000, 32800, 32
    x = torch.zeros(S, K, device="cuda", dtype=torch.uint8)
    x[-300:, 0] = 0x38  # 1.0
    w = torch.zeros(1, N, K, device="cuda", dtype=torch.uint8)
    w[0, :, 0] = torch.where(torch.arange(N, device="cuda") % 2 == 0, 0x38, 0x40).to(torch.uint8)  # 1.0, 2.0
    atoms = torch.full((bsmm.scale_atoms_size(1, N, K),), 127, device="cuda", dtype=torch.uint8)
    y = bsmm.expert_gemm(x, torch.full((S, 1), 127, device="cuda", dtype=torch.uint8), w, atoms, offsets_of([S]))
    assert bool((y[-300:, ::2] == 1).all()) and bool((y[-300:, 1::2] == 2).all()) and not bool(y[-400:-300].any())


def backward_inputs(counts, N, K, rows, seed=0):
    E, S = len(counts), int(sum(counts))
    g = torch.Generator("cuda").manual_seed(seed + S + 3 * N + K)
    X = max(S, 1) if rows is None else rows

    def rnd(*s):
        return (torch.randn(*s, device="cuda", generator=g) * torch.exp2(torch.randint(-4, 5, s, device="cuda", generator=g).float())).bfloat16()

    r = None if rows is None else torch.randint(0, X, (S,), device="cuda", generator=g, dtype=torch.int32)
    return rnd(X if rows is None else S, N), rnd(E, N, K), rnd(X, K), r


BACKWARD = [([1], 32, 32, None), ([3, 0], 64, 96, 2), ([32, 31, 33], 160, 64, None), ([128, 127, 129, 0, 1], 96, 288, 50),
            ([300, 20], 288, 320, 200), ([5, 0, 0, 250, 90], 416, 544, None), ([0, 0], 64, 32, None),
            ([600, 500], 640, 768, 900), ([9] * 20, 256, 128, 30), ([2, 700], 1312, 160, None)]


@pytest.mark.parametrize("counts,N,K,rows", BACKWARD)
@pytest.mark.parametrize("fp8", ["e5m2", "e4m3"])
def test_backward(counts, N, K, rows, fp8):
    bsmm = _bsmm()
    dY, W, X, r = backward_inputs(counts, N, K, rows)
    off = offsets_of(counts)
    S, E = dY.shape[0], len(counts)
    dX = torch.full((S, K), 5.0, device="cuda").bfloat16()
    dW = torch.full((E, N, K), float("nan"), device="cuda").bfloat16()
    ws = torch.full((bsmm.expert_backward_workspace_size(S, E, N, K),), 0xFF, dtype=torch.uint8, device="cuda")
    bsmm.expert_backward(dY, W, X, off, rows=r, fp8=fp8, dX=dX, dW=dW, workspace=ws)
    rX, rW, mX, mW = O.backward(dY.float().cpu().numpy(), W.float().cpu().numpy(), X.float().cpu().numpy(),
                                off.cpu().numpy(), None if r is None else r.cpu().numpy(), fp8)
    check(dX, rX, mX, N, left=5.0)
    check(dW, rW, mW, max(max(counts), 1))
    assert bsmm.check_device_status()[0] == 0


def test_backward_slots_of_no_expert():
    bsmm = _bsmm()
    dY, W, X, r = backward_inputs([40, 60], 96, 64, 30)
    dY[:10] = float("nan")  # padding's gradients are whatever they are
    dY[75:] = float("nan")
    off = torch.tensor([10, 42, 75], dtype=torch.int32, device="cuda")
    dX, dW = bsmm.expert_backward(dY, W, X, off, rows=r, dX=torch.full((100, 64), 1.5, device="cuda").bfloat16())
    rX, rW, mX, mW = O.backward(np.nan_to_num(dY.float().cpu().numpy()), W.float().cpu().numpy(),
                                X.float().cpu().numpy(), off.cpu().numpy(), r.cpu().numpy(), "e5m2")
    check(dX, rX, mX, 96, left=1.5)
    check(dW, rW, mW, 33)


def test_backward_one_after_another():
    """Calls that share a workspace, each overlapping the end of the one before."""
    bsmm = _bsmm()
    sets = [backward_inputs(c, 160, 288, 50, seed=i) + (offsets_of(c),)
            for i, c in enumerate(([130, 0, 70, 33], [3, 200, 1, 29], [0, 0, 233, 0]))]
    alone = []
    for dY, W, X, r, off in sets:
        alone.append([t.clone() for t in bsmm.expert_backward(dY, W, X, off, rows=r)])
        torch.cuda.synchronize()
    ws = torch.empty(bsmm.expert_backward_workspace_size(233, 4, 160, 288), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(30):
        dY, W, X, r, off = sets[i % 3]
        dX, dW = bsmm.expert_backward(dY, W, X, off, rows=r, workspace=ws)
        got.append((dX + 0, dW + 0))  # read by the next kernel of the stream
    for i, (dX, dW) in enumerate(got):
        assert torch.equal(dX, alone[i % 3][0]) and torch.equal(dW, alone[i % 3][1]), i


def test_backward_without_slots():
    bsmm = _bsmm()
    W = torch.randn(3, 64, 32, device="cuda").bfloat16()
    e = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    dX, dW = bsmm.expert_backward(e, W, torch.empty(0, 32, device="cuda", dtype=torch.bfloat16), offsets_of([0, 0, 0]))
    assert dX.shape == (0, 32) and not dW.any()


@pytest.mark.parametrize("rows", [None, 21])
def test_gradients_are_the_forwards_differences(rows):
    """On numbers that MXFP8 and bfloat16 hold exactly (0, +-1, +-2, sums below
    256), y is linear in x and in W without any rounding: <dY, y(x + d) - y(x)> =
    <dX, d>, and the same for W."""
    bsmm = _bsmm()
    counts, N, K = [10, 0, 33, 5], 32, 32
    S, E = sum(counts), len(counts)
    X = S if rows is None else rows
    g = torch.Generator("cuda").manual_seed(3)

    def small(*s):
        v = torch.randint(-2, 3, s, device="cuda", generator=g)
        return torch.where(torch.rand(s, device="cuda", generator=g) < 0.3, v, torch.zeros_like(v)).bfloat16()

    off = offsets_of(counts)
    r = None if rows is None else torch.randint(0, X, (S,), device="cuda", generator=g, dtype=torch.int32)
    x, W, dY, dx, dw = small(X, K), small(E, N, K), small(S, N), small(X, K), small(E, N, K)

    def y(x, W):
        xq, xs = bsmm.quantize(x, (1, 32), "e4m3", "ue8m0")
        wq, wa = bsmm.quantize_atoms(W.view(E * N, K), batches=E)
        return bsmm.expert_gemm(xq, xs, wq.view(E, N, K), wa, off, rows=r).double()

    dX, dW = bsmm.expert_backward(dY, W, x, off, rows=r, fp8="e4m3")
    at = torch.arange(S, device="cuda") if r is None else r.long()
    moved = (dY.double() * (y(x + dx, W) - y(x, W))).sum()
    assert float(moved) == float((dX.double() * dx[at].double()).sum())
    assert float((dY.double() * (y(x, W + dw) - y(x, W))).sum()) == float((dW.double() * dw.double()).sum())
