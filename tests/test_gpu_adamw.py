"""bsmm_adamw against its definition: bit for bit in binary32 (every operation
rounded on its own), and against the textbook form in float64.

Against float64: m and v are sums of two products (four roundings: 4 2^-24 of
the magnitudes; v's terms are positive).  The move's relative error is v's half,
m's, and six roundings; p adds two.  Cancellation in m is bounded by the
magnitudes of its two terms."""

import numpy as np
import pytest
import torch

from oracle import adamw as O

pytestmark = pytest.mark.gpu
ARGS = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def rnd(n, seed, scale, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * scale).to(dtype).cuda()


SIZES = [1, 5, 127, 128, 129, 1000, 4095, 4096, 4097, 8192, 12345, 0, 40000]


def tensors(sizes, p=torch.float32, g=torch.float32, bits8=False):
    d = {"params": [rnd(n, 10 * n + 1, 0.02, p) for n in sizes], "grads": [rnd(n, 10 * n + 2, 1e-3, g) for n in sizes],
         "m": [rnd(n, 10 * n + 3, 3e-4) for n in sizes], "v": [rnd(n, 10 * n + 4, 1e-3).square() for n in sizes]}
    if bits8:
        for name in ("m", "v"):
            x = [t.cpu().numpy() for t in d[name]]
            x = [np.sqrt(t) for t in x] if name == "v" else x
            s = [O.scales(t) for t in x]
            d[name] = [torch.from_numpy(O.codes(t, q, name == "v")).cuda() for t, q in zip(x, s)]
            d[name + "_scales"] = [torch.from_numpy(q[:(t.size + 127) // 128]).cuda() for t, q in zip(x, s)]
    return d


def np32(t):
    return t.detach().float().cpu().numpy()


def expected(d, i, bits8, step, scale=1.0):
    m, v = d["m"][i], d["v"][i]
    if bits8:
        m = O.values(m.cpu().numpy(), np32(d["m_scales"][i]))
        v = O.values(v.cpu().numpy(), np32(d["v_scales"][i]))
        v = (v * v).astype(np.float32)
    else:
        m, v = np32(m), np32(v)
    return (np32(d["params"][i]), np32(d["grads"][i]), m, v), O.step32(np32(d["params"][i]), np32(d["grads"][i]), m, v, step,
                                                                     grad_scale=scale, **ARGS)


def same(t, x):
    """Equal as the tensor's type holds x."""
    return torch.equal(t, torch.from_numpy(np.ascontiguousarray(x)).cuda().to(t.dtype))


@pytest.mark.parametrize("p", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("copies", [False, True])
def test_step(p, g, bits8, copies):
    d = tensors(SIZES, p, g, bits8)
    want = [expected(d, i, bits8, 7, 0.5)[1] for i in range(len(SIZES))]
    cc = [torch.zeros(n, device="cuda", dtype=torch.bfloat16) for n in SIZES] if copies else None
    _bsmm().adamw(d["params"], d["grads"], d["m"], d["v"], 7, grad_scale=0.5, m_scales=d.get("m_scales"),
                  v_scales=d.get("v_scales"), copies=cc, **ARGS)
    for i, n in enumerate(SIZES):
        wp, wm, wv = want[i]
        assert same(d["params"][i], wp), n
        if copies:
            assert same(cc[i], wp), n
        if bits8:
            for name, x, root in (("m", wm, False), ("v", np.sqrt(wv), True)):
                s = O.scales(x)[:(n + 127) // 128]
                assert same(d[name + "_scales"][i], s), (n, name)
                assert same(d[name][i], O.codes(x, s, root)), (n, name)
        else:
            assert same(d["m"][i], wm) and same(d["v"][i], wv), n


@pytest.mark.parametrize("step", [1, 2, 1000, 10 ** 7])
def test_against_the_textbook(step):
    d = tensors([5000])
    (p, g, m, v), _ = expected(d, 0, False, step)
    _bsmm().adamw(d["params"], d["grads"], d["m"], d["v"], step, **ARGS)
    wp, wm, wv = O.step(p, g, m, v, step, **ARGS)
    U = 2.0 ** -24
    mag = 0.9 * np.abs(m) + 0.1 * np.abs(g)
    assert (np.abs(np32(d["m"][0]) - wm) <= 4 * U * mag).all()
    assert (np.abs(np32(d["v"][0]) - wv) <= 5 * U * wv).all()
    bias1, bias2 = 1 - 0.9 ** step, 1 - 0.95 ** step
    move = 3e-3 * (mag / bias1) / (np.sqrt(wv / bias2) + 1e-8)
    assert (np.abs(np32(d["params"][0]) - wp) <= 16 * U * move + 4 * U * np.abs(p)).all()


def test_a_lost_second_moment_keeps_its_smallest_code():
    """Roots far below their block's largest: none becomes zero, and a tensor of
    zeros stays one."""
    n = 256
    root = np.full(n, 1e-9, np.float32)
    root[0] = 1.0
    root[128:] = 0.0
    g, m = np.zeros(n, np.float32), np.zeros(n, np.float32)
    s = O.scales(root)
    d = {"v": O.codes(root, s, True), "m": O.codes(m, O.scales(m)), "vs": s, "ms": O.scales(m)}
    d = {k: torch.from_numpy(x).cuda() for k, x in d.items()}
    p = torch.ones(n, device="cuda")
    for step in range(1, 6):
        _bsmm().adamw([p], [torch.from_numpy(g).cuda()], [d["m"]], [d["v"]], step, m_scales=[d["ms"]],
                      v_scales=[d["vs"]], **ARGS)
    assert bool((d["v"][1:128] == 1).all()) and not d["v"][128:].any() and float(d["vs"][1]) == 1.0
    assert bool(torch.isfinite(p).all())


@pytest.mark.parametrize("bits8", [False, True])
def test_tensors_that_are_not_aligned(bits8):
    """Views that start anywhere give the bits of aligned copies."""
    sizes = [9000, 4096, 300]
    d = tensors(sizes, torch.float32, torch.bfloat16, bits8)

    def shifted(ts, by):
        out = []
        for t in ts:
            flat = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
            flat[by:] = t
            out.append(flat[by:])
        return out

    e = {k: shifted(ts, 1) for k, ts in d.items()}
    for x in (d, e):
        _bsmm().adamw(x["params"], x["grads"], x["m"], x["v"], 3, m_scales=x.get("m_scales"), v_scales=x.get("v_scales"),
                      **ARGS)
    for k in d:
        for a, b in zip(d[k], e[k]):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("count", [96, 97, 250, 900])
def test_more_tensors_than_a_launch_takes(count):
    sizes = [1 + (i * 37) % 300 for i in range(count)]
    d = tensors(sizes)
    want = [expected(d, i, False, 4)[1] for i in range(len(sizes))]
    _bsmm().adamw(d["params"], d["grads"], d["m"], d["v"], 4, **ARGS)
    for i in range(len(sizes)):
        assert same(d["params"][i], want[i][0]) and same(d["m"][i], want[i][1])


@pytest.mark.parametrize("bits8", [False, True])
def test_blocks_that_take_several_chunks(bits8):
    """Large, small and ragged tensors in turn under the same blocks."""
    sizes = [1500000, 5, 700001, 2048, 1000003, 4096, 300]
    d = tensors(sizes, torch.float32, torch.bfloat16, bits8)
    want = [expected(d, i, bits8, 9)[1] for i in range(len(sizes))]
    _bsmm().adamw(d["params"], d["grads"], d["m"], d["v"], 9, m_scales=d.get("m_scales"), v_scales=d.get("v_scales"), **ARGS)
    for i in range(len(sizes)):
        wp, wm, wv = want[i]
        assert same(d["params"][i], wp), sizes[i]
        if bits8:
            for name, x, root in (("m", wm, False), ("v", np.sqrt(wv), True)):
                s = O.scales(x)[:(sizes[i] + 127) // 128]
                assert same(d[name + "_scales"][i], s) and same(d[name][i], O.codes(x, s, root)), (sizes[i], name)
        else:
            assert same(d["m"][i], wm) and same(d["v"][i], wv), sizes[i]


def test_lists_that_do_not_fit():
    bsmm = _bsmm()
    kw = dict(step=1, lr=0.1)

    def z(*sizes):
        return [torch.zeros(n, device="cuda") for n in sizes]

    p = z(6, 200)
    with pytest.raises(ValueError, match="CUDA tensors on the current device"):
        bsmm.adamw(p, z(6) + [torch.zeros(200)], z(6, 200), z(6, 200), **kw)
    with pytest.raises(ValueError, match="contiguous"):
        bsmm.adamw(p, [torch.zeros(12, device="cuda")[::2], *z(200)], z(6, 200), z(6, 200), **kw)
    with pytest.raises(ValueError, match=r"m\[1\] holds 199"):
        bsmm.adamw(p, z(6, 200), z(6, 199), z(6, 200), **kw)
    with pytest.raises(ValueError, match="v holds 3 tensors"):
        bsmm.adamw(p, z(6, 200), z(6, 200), z(6, 200, 1), **kw)
    with pytest.raises(ValueError, match="one type"):
        bsmm.adamw(p, [p[0], p[1].bfloat16()], z(6, 200), z(6, 200), **kw)
    with pytest.raises(ValueError, match="1-byte"):
        bsmm.adamw(p, z(6, 200), z(6, 200), z(6, 200), m_scales=z(1, 2), v_scales=z(1, 2), **kw)
    with pytest.raises(TypeError, match="Tensors"):
        bsmm.adamw(p, [p[0], 1.0], z(6, 200), z(6, 200), **kw)
    codes = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (6, 200)]
    with pytest.raises(ValueError, match=r"v_scales\[1\] holds 1 numbers, 2 needed"):
        bsmm.adamw(p, z(6, 200), codes, codes, m_scales=z(1, 2), v_scales=z(1, 1), **kw)
    assert not any(t.any() for t in p)


def test_parameters_and_tuples():
    """Parameters (which require gradients) and any sequence of tensors."""
    a = [torch.nn.Parameter(torch.ones(300, device="cuda")), torch.nn.Parameter(torch.ones(20, 10, device="cuda"))]
    g = tuple(torch.ones_like(t) for t in a)
    _bsmm().adamw(iter(a), g, [torch.zeros_like(t) for t in g], [torch.zeros_like(t) for t in g], 1, lr=0.5, weight_decay=0.0)
    for t in a:
        assert torch.equal(t.detach(), torch.full_like(t, 0.5))


def test_schedule_on_the_device_and_in_a_graph():
    """A captured step takes lr, step and grad_scale from `hyper` at each replay."""
    bsmm = _bsmm()
    a, b = tensors([5000, 77]), tensors([5000, 77])
    hyper = torch.zeros(3, device="cuda")
    rest = {k: v for k, v in ARGS.items() if k != "lr"}
    bsmm.adamw([], [], [], [], 1, lr=0.1)  # nothing to do
    c = tensors([10])  # the library's set-up on a device is not part of a capture
    bsmm.adamw(c["params"], c["grads"], c["m"], c["v"], 1, **ARGS)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bsmm.adamw(b["params"], b["grads"], b["m"], b["v"], 1, lr=9.0, hyper=hyper, **rest)
    for step, lr, scale in ((1, 2.0 ** -9, 1.0), (2, 2.0 ** -8, 0.25), (3, 2.0 ** -10, 2.0)):  # binary32 holds these lr
        bsmm.adamw(a["params"], a["grads"], a["m"], a["v"], step, lr=lr, grad_scale=scale, **rest)
        hyper.copy_(torch.tensor([lr, step, scale]))
        graph.replay()
        for k in a:
            for x, y in zip(a[k], b[k]):
                torch.testing.assert_close(x, y, rtol=2 ** -21, atol=1e-9)  # the device's pow and the host's


def test_large_tensor():
    """More than 2^31 numbers: the last ones move too."""
    n = 2 ** 31 + 4096 + 7
    p = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    m, v = (torch.zeros(n, device="cuda", dtype=torch.uint8) for _ in range(2))
    ms, vs = (torch.ones((n + 127) // 128, device="cuda") for _ in range(2))
    _bsmm().adamw([p], [g], [m], [v], 1, lr=0.25, weight_decay=0.0, m_scales=[ms], v_scales=[vs])
    for at in (0, 2 ** 31 - 1, 2 ** 31, n - 8, n - 1):
        assert float(p[at]) == 0.75, at
    assert bool((m[-1000:] == 0x7E).all()) and bool((v[-1000:] == 0x7E).all())
