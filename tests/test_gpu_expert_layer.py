"""The calls of a mixture of experts together, as a layer uses them: against
autograd in float64 on unquantized operands, inside CUDA graphs whose inputs
change between replays, on other streams and from several host threads.

Tolerances.  E4M3 keeps 3 mantissa bits: a value's relative error is uniform up
to 2^-4, 0.026 root mean square over a binade, and independent from element to
element, so a contraction of two quantized operands is off by 0.026 sqrt(2) =
0.037 of its norm; E5M2 (2 bits) doubles its operand's share: sqrt(0.026^2 +
0.052^2) = 0.058, and 0.052 sqrt(2) = 0.074 with both in E5M2.  A gradient passes
at most two such backward products and the forward's three quantized activations:
sqrt(2 * 0.074^2 + 2 * 0.037^2 + 0.01^2) = 0.12, taken twice for the
nonlinearity: 0.24.  The output passes two forward products: sqrt(2) * 0.037 =
0.053, taken twice: 0.11."""

import importlib.util
import os
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _example():
    spec = importlib.util.spec_from_file_location("expert_mlp", os.path.join(ROOT, "examples", "expert_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,experts,top", [(96, 4, 2), (700, 6, 3), (2048, 16, 1)])
def test_step_against_autograd(tokens, experts, top):
    mlp = _example().make(256, 384, experts, top, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, dy = (torch.randn(tokens, 256, device="cuda", generator=g).bfloat16() for _ in range(2))
    y, saved = mlp.forward(x)
    got = mlp.backward(dy, saved)

    leaves = [t.double().requires_grad_() for t in (x, *mlp.copies)]
    lx, wr, w1, w2 = leaves
    ids = saved[3].long()
    # the choice is the library's own; the router's weights of top = 1 are constant
    p = torch.softmax((lx @ wr.T).gather(1, ids), 1)
    want = 0
    for j in range(top):
        up = torch.einsum("tnd,td->tn", w1[ids[:, j]], lx)
        gate, u = up.chunk(2, dim=1)
        want = want + p[:, j:j + 1] * torch.einsum("tdi,ti->td", w2[ids[:, j]], torch.nn.functional.silu(gate) * u)
    want.backward(dy.double())
    assert _rel(y, want.detach()) < 0.11
    for name, g1, leaf in zip(("dx", "dwr", "dw1", "dw2"), got, leaves):
        if name != "dwr" or top > 1:
            assert _rel(g1, leaf.grad) < 0.24, name
        else:
            assert not g1.any()
    before = [t.clone() for t in mlp.masters]
    mlp.update(got[1:])
    for a, b, c in zip(before, mlp.masters, mlp.copies):
        assert bool(torch.isfinite(b).all()) and torch.equal(c, b.bfloat16())
        assert float((a - b).abs().max()) <= 1.2e-3  # the first step's move is lr, and the decay's share
    assert _bsmm().check_device_status()[0] == 0


@pytest.mark.parametrize("tokens", [5, 129, 900])
def test_captured_step_follows_its_inputs(tokens):
    """One capture, replayed on other tokens (other segment lengths), gives the
    eager calls' bits: nothing of the layout is kept from the capture."""
    mlp = _example().make(256, 128, 8, 2, seed=3)
    x = torch.randn(tokens, 256, device="cuda").bfloat16()
    dy = torch.randn(tokens, 256, device="cuda").bfloat16()

    def step():
        y, saved = mlp.forward(x)
        return (y, *mlp.backward(dy, saved))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(tokens, 256, device="cuda", generator=g))
        if seed == 2:
            x[:] = x[:1]  # all tokens at the same experts, the others empty
        dy.copy_(torch.randn(tokens, 256, device="cuda", generator=g))
        graph.replay()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    assert _bsmm().check_device_status()[0] == 0


def _calls():
    """name -> a call on `stream` (None: the current one)."""
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*s, dtype=torch.bfloat16):
        return torch.randn(*s, device="cuda", generator=g).to(dtype)

    T, k, E, N, K = 500, 3, 7, 160, 256
    l, few = rnd(T, E, dtype=torch.float32), rnd(20, E, dtype=torch.float32)
    w, ids, offsets, rows, slots = bsmm.route(l, k)
    dw = rnd(T, k, dtype=torch.float32)
    xv, W, dY = rnd(T, K), rnd(E, N, K), rnd(T * k, N)
    x, xs = bsmm.quantize(xv, (1, 32), "e4m3", "ue8m0")
    wq, wa = bsmm.quantize_atoms(W.view(E * N, K), batches=E)
    d = rnd(T, N)
    return {"route": lambda s: bsmm.route(l, k, stream=s), "route few": lambda s: bsmm.route(few, k, stream=s),
            "route_backward": lambda s: bsmm.route_backward(dw, l, ids, w, renormalize=False, stream=s),
            "expert_gemm": lambda s: bsmm.expert_gemm(x, xs, wq.view(E, N, K), wa, offsets, rows=rows, stream=s),
            "expert_backward": lambda s: bsmm.expert_backward(dY, W, xv, offsets, rows=rows, stream=s),
            "expert_combine": lambda s: bsmm.expert_combine(dY, slots, w, stream=s),
            "expert_combine_backward": lambda s: bsmm.expert_combine_backward(d, dY, slots, w, stream=s)}


NAMES = ["route", "route few", "route_backward", "expert_gemm", "expert_backward", "expert_combine",
         "expert_combine_backward"]


@pytest.fixture(scope="module")
def made():
    c = _calls()
    torch.cuda.synchronize()
    return c


def _tensors(v):
    return [v] if isinstance(v, torch.Tensor) else list(v)


@pytest.mark.parametrize("name", NAMES)
def test_beside_late_work_of_the_current_stream(made, name):
    ref = [t.clone() for t in _tensors(made[name](None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    late = [torch.empty(t.numel() * t.element_size(), dtype=torch.uint8, device="cuda") for t in ref for _ in range(2)]
    late.append(torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    for t in late:
        t.fill_(0xFF)
    del late, t
    got = _tensors(made[name](s))
    s.synchronize()
    torch.cuda.synchronize()
    for p, q in zip(ref, got):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_the_same_bits_again_and_from_threads(made, name):
    ref = [t.clone() for t in _tensors(made[name](None))]
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(10):
            got = _tensors(made[name](s))
            s.synchronize()
            if not all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(ref, got)):
                bad.append(name)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


MARGIN, SENTINEL = 1 << 16, 0xA5


class Guarded:
    """A tensor inside a sentinel-filled buffer."""

    def __init__(self, shape, dtype):
        n = torch.Size(shape).numel()
        self.nbytes = n * torch.empty((), dtype=dtype).element_size()
        self.buf = torch.full((2 * MARGIN + self.nbytes,), SENTINEL, dtype=torch.uint8, device="cuda")
        self.t = self.buf[MARGIN:MARGIN + self.nbytes].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        assert bool((self.buf[:MARGIN] == SENTINEL).all()) and bool((self.buf[MARGIN + self.nbytes:] == SENTINEL).all())


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 32, 32), (37, 2, 5, 96, 160), (130, 4, 9, 288, 544), (700, 1, 3, 544, 96)])
def test_nothing_is_written_outside(T, k, E, N, K):
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(T)
    S, b16, i32, f32 = T * k, torch.bfloat16, torch.int32, torch.float32

    def rnd(*s):
        return torch.randn(*s, device="cuda", generator=g).bfloat16()

    l = rnd(T, E).float()
    l[0, 0] = -float("inf")
    w, ids, off, rows, slots = (Guarded(s, t) for s, t in (((T, k), f32), ((T, k), i32), ((E + 1,), i32), ((S,), i32), ((T, k), i32)))
    ws = Guarded((max(bsmm.route_workspace_size(T, E), 256),), torch.uint8)
    bsmm.route(l, k, weights=w.t, ids=ids.t, offsets=off.t, rows=rows.t, slots=slots.t, workspace=ws.t)
    dl = Guarded((T, E), f32)
    bsmm.route_backward(torch.ones(T, k, device="cuda"), l, ids.t, w.t, renormalize=False, d_logits=dl.t)
    xv, W, dY = rnd(T, K), rnd(E, N, K), rnd(S, N)
    x, xs = bsmm.quantize(xv, (1, 32), "e4m3", "ue8m0")
    wq, wa = bsmm.quantize_atoms(W.view(E * N, K), batches=E)
    y = Guarded((S, N), b16)
    gw = Guarded((max(bsmm.expert_gemm_workspace_size(S, E, K), 256),), torch.uint8)
    bsmm.expert_gemm(x, xs, wq.view(E, N, K), wa, off.t, rows=rows.t, y=y.t, workspace=gw.t)
    dX, dW = Guarded((S, K), b16), Guarded((E, N, K), b16)
    bw = Guarded((bsmm.expert_backward_workspace_size(S, E, N, K),), torch.uint8)
    bsmm.expert_backward(dY, W, xv, off.t, rows=rows.t, dX=dX.t, dW=dW.t, workspace=bw.t)
    out, dy, dw = Guarded((T, N), b16), Guarded((S, N), b16), Guarded((T, k), f32)
    bsmm.expert_combine(y.t, slots.t, w.t, out=out.t)
    bsmm.expert_combine_backward(rnd(T, N), y.t, slots.t, w.t, dy=dy.t, d_weights=dw.t)
    for m in (w, ids, off, rows, slots, ws, dl, y, gw, dX, dW, bw, out, dy, dw):
        m.check()
    n = 5 * T + 3
    ts = [Guarded((n,), t) for t in (f32, b16, torch.uint8, torch.uint8, b16)]
    scales = [Guarded(((n + 127) // 128,), f32) for _ in range(2)]
    for t in ts[:2] + scales:
        t.t.fill_(1.0)
    for t in ts[2:4]:
        t.t.zero_()
    bsmm.adamw([ts[0].t], [ts[1].t], [ts[2].t], [ts[3].t], 1, lr=0.1, m_scales=[scales[0].t], v_scales=[scales[1].t],
               copies=[ts[4].t])
    for m in ts + scales:
        m.check()
    assert bsmm.check_device_status()[0] == 0
