"""bsmm_adamw's 8-bit states over many steps: beside binary32 states, bit for bit
against their definition where they are dithered, and the same bits again.

The tolerance over many steps is derived in test_state_dither."""

import numpy as np
import pytest
import torch

from oracle import adamw as O
from test_state_dither import states_tolerance

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def rnd(n, seed, scale, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * scale).to(dtype).cuda()


def np32(t):
    return t.detach().float().cpu().numpy()


def states(n, seed=0):
    """Codes and scales of states in mid-run."""
    m, root = np32(rnd(n, seed + 1, 3e-4)), np.abs(np32(rnd(n, seed + 2, 1e-3)))
    s, q = O.scales(m), O.scales(root)
    blocks = (n + 127) // 128
    return [torch.from_numpy(x).cuda() for x in (O.codes(m, s), O.codes(root, q, True), s[:blocks], q[:blocks])]


def values(codes, scales):
    return O.values(codes.cpu().numpy(), np32(scales))


def run(betas, steps, gradients, numbers=1024):
    """The parameters and states after the steps, binary32 and in 8 bits."""
    bsmm = _bsmm()
    z = lambda dtype=torch.float32, n=numbers: torch.zeros(n, dtype=dtype, device="cuda")  # noqa: E731
    p, m, v = z(), z(), z()
    p8, m8, v8, ms, vs = z(), z(torch.uint8), z(torch.uint8), z(n=(numbers + 127) // 128), z(n=(numbers + 127) // 128)
    kw = dict(lr=1e-3, betas=betas, weight_decay=0.0)
    for t in range(1, steps + 1):
        g = gradients(t)
        bsmm.adamw([p], [g], [m], [v], t, **kw)
        bsmm.adamw([p8], [g], [m8], [v8], t, m_scales=[ms], v_scales=[vs], **kw)
    return (np32(p), np32(m), np.sqrt(np32(v))), (np32(p8), m8, v8, ms, vs)


@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.9, 0.99), (0.95, 0.97)])
def test_states_follow_gradients_that_fall(betas):
    """From step 300 on every second number's gradients are a twentieth."""
    g = torch.Generator(device="cuda").manual_seed(7)
    low = torch.arange(1024, device="cuda") % 2 == 0

    def gradients(t):
        x = torch.randn(1024, device="cuda", generator=g) * 1e-3
        return torch.where(low, x * 0.05, x) if t > 300 else x

    (_, _, root), (_, _, v8, _, vs) = run(betas, 700, gradients)
    r = values(v8, vs) / root
    mean, sd = states_tolerance(512)
    for half in (r[::2], r[1::2]):
        assert abs(half.mean() - 1) <= mean and np.sqrt(np.mean((half - 1) ** 2)) <= sd + mean


def test_numbers_whose_gradients_end_stop():
    """0.9^300 of a first moment is 2e-14 of it, below every number above zero that
    its codes have (2^-9 / 448 of the block's largest): the mean is kept only by
    codes of zero.  Its parameter then keeps its place."""
    g = torch.Generator(device="cuda").manual_seed(8)
    idle = torch.arange(1024, device="cuda") % 2 == 0

    def gradients(t):
        x = torch.randn(1024, device="cuda", generator=g) * 1e-3
        return torch.where(idle, torch.zeros_like(x), x) if t > 100 else x

    _, (_, m8, _, _, _) = run((0.9, 0.999), 400, gradients)
    assert not (m8[idle] & 0x7F).any() and bool((m8[~idle] & 0x7F).any())


@pytest.mark.parametrize("p", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("g", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("betas", [(0.9, 0.999), (0.97, 0.95), (0.9, 0.96)])
@pytest.mark.parametrize("off", [0, 1])
def test_bits(p, g, betas, off):
    """Large and ragged tensors, aligned and not, one list."""
    assert O.dithers(betas)
    bsmm = _bsmm()
    sizes = [1, 5, 127, 128, 129, 2048, 4097, 0, 300001]

    def shifted(t):
        flat = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
        flat[off:] = t
        return flat[off:]

    ps, gs = [shifted(rnd(n, n + 1, 0.02, p)) for n in sizes], [shifted(rnd(n, n + 2, 1e-3, g)) for n in sizes]
    ms, vs, mss, vss = ([shifted(t) for t in ts] for ts in zip(*(states(n, n) for n in sizes)))
    kw = dict(lr=3e-3, betas=betas, eps=1e-8, weight_decay=0.1)
    want = []
    for i in range(len(sizes)):
        root = values(vs[i], vss[i])
        want.append(O.step32(np32(ps[i]), np32(gs[i]), values(ms[i], mss[i]), root * root, 12345, **kw))
    bsmm.adamw(ps, gs, ms, vs, 12345, m_scales=mss, v_scales=vss, **kw)
    for i, n in enumerate(sizes):
        wp, wm, wv = want[i]
        assert torch.equal(ps[i], torch.from_numpy(wp).cuda().to(p)), n
        for codes, scales, x, root in ((ms[i], mss[i], wm, False), (vs[i], vss[i], np.sqrt(wv), True)):
            s = O.scales(x)[:(n + 127) // 128]
            np.testing.assert_array_equal(np32(scales), s)
            np.testing.assert_array_equal(codes.cpu().numpy(), O.codes(x, s, root, step=12345))


def test_a_captured_schedule_dithers_by_its_step():
    """The same bits as eager steps, replay by replay, and others for other steps."""
    bsmm = _bsmm()
    n, rest = 5000, dict(betas=(0.9, 0.999), weight_decay=0.0)
    g = rnd(n, 1, 1e-3)
    a, b = ([torch.zeros(n, device="cuda"), *states(n)] for _ in range(2))
    hyper = torch.zeros(3, device="cuda")

    def step(x, t, **kw):
        bsmm.adamw([x[0]], [g], [x[1]], [x[2]], t, m_scales=[x[3]], v_scales=[x[4]], **rest, **kw)

    c = [torch.zeros(n, device="cuda"), *states(n)]
    step(c, 1, lr=0.1)  # the library's set-up on a device is not part of a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b, 1, lr=9.0, hyper=hyper)
    for t in (1, 2, 70000):
        before = a[2].clone()
        step(a, t, lr=2.0 ** -9)
        hyper.copy_(torch.tensor([2.0 ** -9, t, 1.0]))
        graph.replay()
        for x, y in zip(a[1:], b[1:]):  # the states do not depend on the factors of lr and of the biases
            assert torch.equal(x, y), t
        again, other = ([c[0].clone(), a[1].clone(), before.clone(), a[3].clone(), a[4].clone()] for _ in range(2))
        step(again, t, lr=0.1)
        step(other, t + 1, lr=0.1)
        assert not torch.equal(again[2], other[2])
