"""bsmm_adapters and bsmm_adapters_backward against their float64 forms.

Tolerances come from the arithmetic.  A product's operands are bfloat16, so
each product is exact in binary32; a sum of n of them in binary32 is off by at
most n 2^-23 of the sum of magnitudes, even if every addition truncates.  u
and d enter the second product as two bfloat16 terms (2^-17 of them is lost)
where the result is bfloat16, as three (2^-24) where it is binary32.  A
bfloat16 result adds half its ulp, 2^-9 of the magnitude's power of two, so at
most 2^-8 of the value."""

import numpy as np
import pytest
import torch

from oracle import adapters as O
from oracle import checkpoint as C

pytestmark = pytest.mark.gpu

E = 2.0 ** -23


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make(T, K, N, R, L, seed=0, ids="mixed", y="bf16"):
    g = torch.Generator().manual_seed(seed * 7919 + T + 3 * K + 5 * N + 7 * R + L)
    rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(torch.bfloat16)  # noqa: E731
    d = {"x": rnd(T, K), "a": rnd(L, R, K, k=K ** -0.5), "b": rnd(L, N, R, k=R ** -0.5), "dy": rnd(T, N),
         "dx_base": rnd(T, K), "scaling": torch.rand(L, generator=g) * 2 - 0.5}
    if ids == "runs":
        i = torch.arange(T) * (L + 1) // max(T, 1) - 1
    elif ids == "none":
        i = torch.full((T,), -1)
    else:
        i = torch.randint(-1, L + 1, (T,), generator=g)  # -1 and L: no adapter
    d["ids"] = i.to(torch.int32)
    if y != "none":
        d["y"] = torch.randn(T, N, generator=g).to(torch.float32 if y == "f32" else torch.bfloat16)
    return d


def cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def check(got, ref, bound, half_ulp, what):
    got = _f64(got)
    tol = bound + half_ulp * np.abs(ref) + 1e-30
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) / tol):.3g} of the tolerance, first at {np.argwhere(bad)[0]}")


def forward_bounds(d, f32):
    x, a, b, ids = (_f64(d[k]) for k in ("x", "a", "b", "ids"))
    K, R, sc = x.shape[1], b.shape[2], _f64(d["scaling"])
    mag_u = O.forward(np.abs(x), np.abs(a), np.abs(b), ids)[1]
    u = O.forward(x, a, b, ids)[1]
    lost = 2.0 ** (-23 if f32 else -17)
    out = np.zeros((x.shape[0], b.shape[1]))
    for t, k in enumerate(ids.astype(int)):
        if 0 <= k < b.shape[0]:
            eu = K * E * mag_u[t] + (lost + R * 3 * E) * np.abs(u[t])
            out[t] = abs(sc[k]) * (np.abs(b[k]) @ eu)
    return out, K * E * mag_u


FORWARD = [  # T, K, N, R, L, ids, y
    (1, 512, 384, 16, 4, "mixed", "bf16"), (1, 8, 8, 1, 1, "runs", "f32"), (1, 4096, 1024, 64, 3, "mixed", "f32"),
    (2, 33, 17, 5, 2, "mixed", "bf16"), (5, 256, 256, 8, 9, "mixed", "none"), (16, 128, 96, 12, 16, "mixed", "f32"),
    (17, 1000, 72, 24, 3, "mixed", "bf16"), (64, 512, 520, 16, 64, "mixed", "bf16"), (63, 264, 200, 33, 7, "mixed", "f32"),
    (129, 160, 136, 128, 2, "runs", "bf16"), (300, 544, 264, 4, 5, "runs", "f32"), (777, 96, 160, 32, 5, "mixed", "bf16"),
    (2048, 264, 136, 16, 3, "runs", "bf16"), (2049, 71, 45, 7, 4, "mixed", "f32"), (2300, 128, 1032, 64, 4, "runs", "f32"),
    (2100, 64, 64, 128, 3, "mixed", "bf16"), (2050, 512, 40, 8, 40, "mixed", "bf16"), (40, 64, 64, 16, 3, "none", "bf16"),
    (2500, 96, 80, 12, 3, "mixed", "f32"), (2200, 72, 328, 24, 4, "runs", "bf16"), (2048, 704, 96, 32, 2, "runs", "none"),
    (8200, 64, 72, 16, 6, "mixed", "bf16"), (2176, 64, 200, 128, 2, "runs", "f32"), (2100, 64, 64, 16, 3, "none", "bf16"),
    (2100, 36, 1000, 16, 1100, "mixed", "bf16"),
    # sorted with a few tokens to a tile, and as they come with many adapters
    (300, 128, 200, 64, 40, "mixed", "bf16"), (260, 201, 136, 128, 12, "mixed", "f32"), (96, 264, 136, 16, 64, "mixed", "f32"),
    (700, 136, 72, 8, 300, "mixed", "f32"), (1500, 72, 99, 16, 200, "mixed", "bf16"),
]


@pytest.mark.parametrize("T,K,N,R,L,ids,y", FORWARD)
def test_forward(T, K, N, R, L, ids, y):
    d = make(T, K, N, R, L, ids=ids, y=y)
    ref, uref = O.forward(*(_f64(d[k]) for k in ("x", "a", "b", "ids")), _f64(d["y"]) if "y" in d else None,
                          _f64(d["scaling"]))
    g = cuda(d)
    out, u = _bsmm().adapters(g["x"], g["a"], g["b"], g["ids"], y=g.get("y"), scaling=g["scaling"])
    f32 = out.dtype == torch.float32
    assert f32 == (y == "f32")
    bo, bu = forward_bounds(d, f32)
    check(u, uref, bu, 0.0, "u")
    check(out, ref, bo, 2.0 ** -23 * 2 if f32 else 2.0 ** -8, "out")


def test_no_scaling_in_place_and_float32_delta():
    d = cuda(make(50, 256, 128, 16, 4))
    bsmm = _bsmm()
    one = torch.ones(4, device="cuda")
    ref, _ = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"], scaling=one)
    y = d["y"].clone()
    out, _ = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=y, out=y)
    assert out is y and torch.equal(out, ref)
    delta, u = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], out_dtype=torch.float32)
    assert delta.dtype == torch.float32
    off = (d["ids"] < 0) | (d["ids"] >= 4)
    assert off.any() and not delta[off].any() and not u[off].any()


@pytest.mark.parametrize("T", [40, 2100])
def test_strided_rows(T):
    """x, y and out as column slices of wider arrays, at aligned and odd offsets."""
    bsmm = _bsmm()
    d = cuda(make(T, 128, 96, 16, 3))
    ref, uref = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"], scaling=d["scaling"])
    for off in (8, 3):
        wide = lambda v: torch.nn.functional.pad(v, (off, 24 - off), value=7.0)  # noqa: E731
        xw, yw = wide(d["x"]), wide(d["y"])
        ow = torch.full_like(yw, 5.0)
        sl = slice(off, off + 96)
        out, u = bsmm.adapters(xw[:, off:off + 128], d["a"], d["b"], d["ids"], y=yw[:, sl], scaling=d["scaling"],
                               out=ow[:, sl])
        assert torch.equal(out, ref) and torch.equal(u, uref)
        assert (ow[:, :off] == 5).all() and (ow[:, off + 96:] == 5).all()


@pytest.mark.parametrize("T", [16, 48, 2112])
def test_rows_do_not_mix(T):
    """An infinity or NaN in one adapter's weights or in one token reaches only
    the rows that use it, forward and backward."""
    bsmm = _bsmm()
    d = cuda(make(T, 96, 64, 16, 4))
    ids = torch.arange(T, device="cuda", dtype=torch.int32) % 5 - 1
    clean = bsmm.adapters(d["x"], d["a"], d["b"], ids, y=d["y"], scaling=d["scaling"])
    args = dict(scaling=d["scaling"], dx_base=d["dx_base"])
    clean_b = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], ids, clean[1], **args)
    a, b, x, dy = d["a"].clone(), d["b"].clone(), d["x"].clone(), d["dy"].clone()
    a[2, 3, 5] = float("nan")
    b[2, 7, 1] = float("inf")
    sick = torch.nonzero(ids == 1)[0, 0]
    x[sick, 11] = float("inf")
    dy[sick, 13] = float("nan")
    x[torch.nonzero(ids == -1)[0, 0]] = float("nan")
    dy[torch.nonzero(ids == -1)[0, 0]] = float("nan")
    out, u = bsmm.adapters(x, a, b, ids, y=d["y"], scaling=d["scaling"])
    well = (ids != 2) & (torch.arange(T, device="cuda") != sick)
    assert torch.equal(out[well], clean[0][well]) and torch.equal(u[well], clean[1][well])
    assert out[ids == 2].isnan().any()
    dx, da, db = bsmm.adapters_backward(dy, x, a, b, ids, clean[1], **args)
    assert torch.equal(dx[well], clean_b[0][well])
    for k in (0, 3):
        assert torch.equal(da[k], clean_b[1][k]) and torch.equal(db[k], clean_b[2][k])
    assert da[1].isnan().any() and db[1].isnan().any()


BACKWARD = [  # T, K, N, R, L, ids, x, grad
    (1, 64, 96, 16, 2, "mixed", "bf16", "f32"), (3, 32, 40, 8, 3, "mixed", "e4m3", "bf16"),
    (17, 33, 17, 5, 2, "mixed", "bf16", "f32"), (64, 256, 264, 16, 1, "runs", "e4m3", "f32"),
    (65, 160, 136, 24, 4, "mixed", "e5m2", "f32"), (200, 136, 520, 4, 3, "runs", "bf16", "bf16"),
    (1333, 72, 64, 12, 3, "mixed", "bf16", "f32"), (700, 128, 96, 128, 2, "runs", "e4m3", "f32"),
    (2100, 96, 72, 64, 2, "runs", "e4m3", "bf16"), (2049, 45, 71, 7, 3, "mixed", "bf16", "f32"),
    (40, 64, 64, 16, 3, "none", "bf16", "f32"), (2060, 264, 200, 33, 5, "mixed", "bf16", "f32"),
    (2304, 288, 320, 32, 2, "runs", "e5m2", "f32"), (8300, 96, 64, 16, 3, "mixed", "e4m3", "f32"),
    (640, 160, 44, 16, 2, "runs", "e4m3", "bf16"), (2200, 72, 64, 24, 300, "mixed", "bf16", "f32"),
    (900, 64, 72, 8, 100, "mixed", "bf16", "f32"), (300, 96, 128, 32, 60, "mixed", "e4m3", "f32"),
    # sums of several rounds
    (16000, 64, 72, 16, 1, "runs", "bf16", "f32"), (27000, 32, 40, 64, 1, "runs", "e4m3", "f32"),
    (16000, 64, 64, 24, 1, "mixed", "e4m3", "f32"), (27000, 32, 40, 128, 1, "mixed", "bf16", "f32"),
]


@pytest.mark.parametrize("T,K,N,R,L,ids,xk,grad", BACKWARD)
def test_backward(T, K, N, R, L, ids, xk, grad):
    bsmm = _bsmm()
    d = make(T, K, N, R, L, ids=ids)
    g = cuda(d)
    x64, kw = _f64(d["x"]), {}
    x = g["x"]
    if xk != "bf16":
        x, xs = bsmm.quantize(g["x"], (1, 32), xk, "ue8m0")
        x64 = C.values(x.cpu().numpy(), xs.cpu().numpy(), xk).astype(np.float64)
        kw = dict(x_scales=xs, x_code=xk)
    a64, b64, i64, s64 = (_f64(d[k]) for k in ("a", "b", "ids", "scaling"))
    u = torch.from_numpy(O.forward(x64, a64, b64, i64)[1]).float()
    u64 = u.numpy().astype(np.float64)
    dy64, base64 = _f64(d["dy"]), _f64(d["dx_base"])
    gd = torch.float32 if grad == "f32" else torch.bfloat16
    dx, da, db = bsmm.adapters_backward(g["dy"], x, g["a"], g["b"], g["ids"], u.cuda(), scaling=g["scaling"],
                                        dx_base=g["dx_base"], grad_dtype=gd, **kw)
    rdx, rda, rdb, rd = O.backward(dy64, x64, a64, b64, i64, u64, base64, s64)
    mag_d = O.backward(np.abs(dy64), np.abs(x64), np.abs(a64), np.abs(b64), i64, np.abs(u64))[3]
    lost = 2.0 ** -17
    ed = N * E * mag_d + (lost + 3 * R * E) * np.abs(rd)  # error of d as dx uses it
    bound = O.backward(np.ones_like(dy64), x64, np.abs(a64), np.zeros_like(b64), i64, u64)[0] * 0
    for t, k in enumerate(i64.astype(int)):
        if 0 <= k < L:
            bound[t] = abs(s64[k]) * (np.abs(a64[k]).T @ ed[t])
    check(dx, rdx, bound, 2.0 ** -8, "dx")
    # gradients: the tokens' sum (T additions of up to 3 terms), d's own error, the terms' loss
    lost = 2.0 ** (-23 if grad == "f32" else -17)
    half = 2.0 ** (-23 if grad == "f32" else -8)
    bda, bdb = np.zeros_like(a64), np.zeros_like(b64)
    for t, k in enumerate(i64.astype(int)):
        if 0 <= k < L:
            s = abs(s64[k])
            bda[k] += s * np.outer(N * E * mag_d[t] + (lost + 3 * T * E) * np.abs(rd[t]), np.abs(x64[t]))
            bdb[k] += s * np.outer(np.abs(dy64[t]), (lost + 3 * T * E) * np.abs(u64[t]))
    check(da, rda, bda, half, "dA")
    check(db, rdb, bdb, half, "dB")


def test_gradients_against_differences():
    """out is linear in x, in A and in B, so with loss = sum(out * dy) the
    difference over a step of one of them is its gradient's product with the
    step, exactly but for rounding."""
    bsmm = _bsmm()
    T, K, N, R, L = 70, 96, 64, 8, 3
    d = cuda(make(T, K, N, R, L))

    def loss(x, a, b):
        return (bsmm.adapters(x, a, b, d["ids"], scaling=d["scaling"], out_dtype=torch.float32)[0].double()
                * d["dy"].double()).sum().item()

    u = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], scaling=d["scaling"], out_dtype=torch.float32)[1]
    dx, da, db = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"], u, scaling=d["scaling"])
    at = loss(d["x"], d["a"], d["b"])
    for name, grad in (("x", dx), ("a", da), ("b", db)):
        step = torch.where(torch.rand_like(d[name].float()) < 0.5, 0.5, -0.5).to(torch.bfloat16)
        moved = (d[name].float() + step.float()).to(torch.bfloat16)
        actual = moved.double() - d[name].double()
        args = {k: moved if k == name else d[k] for k in ("x", "a", "b")}
        diff = loss(**args) - at
        predicted = (grad.double() * actual).sum().item()
        scale = (grad.double().abs() * actual.abs()).sum().item()
        # dx is bfloat16 (2^-9 of each term, random signs: well below 2^-9 of the sum of magnitudes)
        assert abs(diff - predicted) <= scale * (2.0 ** -9 if name == "x" else 1e-5), (name, diff, predicted)


def test_empty_and_unused():
    bsmm = _bsmm()
    d = cuda(make(8, 64, 32, 16, 3))
    out, u = bsmm.adapters(d["x"][:0], d["a"], d["b"], d["ids"][:0], y=d["y"][:0])
    assert out.shape == (0, 32) and u.shape == (0, 16)
    da = torch.full((3, 16, 64), 9.0, device="cuda")
    dx, da, db = bsmm.adapters_backward(d["dy"][:0], d["x"][:0], d["a"], d["b"], d["ids"][:0], u, da=da)
    assert dx.shape == (0, 64) and not da.any() and not db.any()
    ids = torch.ones(8, dtype=torch.int32, device="cuda")
    u = torch.randn(8, 16, device="cuda")
    _, da, db = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], ids, u)
    for g in (da, db):
        assert g[1].any() and not g[0].any() and not g[2].any()


def test_stream_graph_and_repeat():
    """The same bits on a stream of its own, in a CUDA graph and again."""
    bsmm = _bsmm()
    d = cuda(make(100, 512, 256, 16, 5))
    ref = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"], scaling=d["scaling"])
    refb = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"], ref[1], scaling=d["scaling"],
                                  dx_base=d["dx_base"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"], scaling=d["scaling"], stream=s)
    gotb = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"], got[1], scaling=d["scaling"],
                                  dx_base=d["dx_base"], stream=s)
    s.synchronize()
    for p, q in zip(ref + refb, got + gotb):
        assert torch.equal(p, q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"], scaling=d["scaling"])
        ob = bsmm.adapters_backward(d["dy"], d["x"], d["a"], d["b"], d["ids"], o[1], scaling=d["scaling"],
                                    dx_base=d["dx_base"])
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(ref + refb, o + ob):
        assert torch.equal(p, q)


def test_offsets_beyond_32_bits():
    """Rows whose byte offset passes 2^32: the last tokens of a strided x and out."""
    bsmm = _bsmm()
    T, K, N, R = 2200, 64, 64, 8
    pitch = 1 << 20  # 2200 rows of 2 MiB each: 4.6 GB
    d = cuda(make(T, K, N, R, 2, ids="runs"))
    xw = torch.empty((T, pitch), dtype=torch.bfloat16, device="cuda")
    xw[:, :K] = d["x"]
    ow = torch.empty((T, pitch), dtype=torch.bfloat16, device="cuda")
    ref, uref = bsmm.adapters(d["x"], d["a"], d["b"], d["ids"], y=d["y"])
    out, u = bsmm.adapters(xw[:, :K], d["a"], d["b"], d["ids"], y=d["y"], out=ow[:, :N])
    assert torch.equal(out, ref) and torch.equal(u, uref)
