"""Calls with ``stream=``: what the binding allocates for them comes from that
stream's own memory pool, so that it is not memory in which earlier work of the
current stream is still under way; and the chains of kernels that run many
tokens give the same bits on another stream, inside a CUDA graph, again, and
from several host threads."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def _tensors(v):
    if isinstance(v, torch.Tensor):
        return [v]
    if isinstance(v, dict):
        v = [v[k] for k in sorted(v)]
    return [t for x in v for t in _tensors(x)] if isinstance(v, (list, tuple)) else []


def calls():
    """name -> a call on `stream` (None: the current one); inputs are made once."""
    bsmm = _bsmm()
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*s, dtype=torch.bfloat16):
        return torch.randn(*s, device="cuda", generator=g).to(dtype)

    T, K, N, R, L = 2100, 256, 384, 16, 5
    x, dy, y = rnd(T, K), rnd(T, N), rnd(T, N)
    a, b = rnd(L, R, K), rnd(L, N, R)
    ids = torch.randint(-1, L, (T,), device="cuda", dtype=torch.int32, generator=g)
    u = rnd(T, R, dtype=torch.float32)
    M, F = 256, 512
    p, w, dyl = rnd(M, F), rnd(N, F), rnd(M, N)
    pq, ps = bsmm.quantize(p, (1, 32), "e4m3", "ue8m0")
    wq, ws = bsmm.quantize(w, (1, 32), "e4m3", "ue8m0")
    gq, gs = bsmm.quantize(p, (1, 128), "e4m3", "f32")
    hq, hs = bsmm.quantize(w, (128, 128), "e4m3", "f32")
    pa, wa = bsmm.quantize_atoms(p), bsmm.quantize_atoms(w)
    n4q, n4s = bsmm.quantize(p, (1, 16), "e2m1", "ue4m3")
    m4q, m4s = bsmm.quantize(w, (1, 16), "e2m1", "ue4m3")
    ops = [t for v in ((dyl, False), (w, True), (dyl, True), (p, True))
           for t in bsmm.quantize_atoms(v[0], code="e5m2", transpose=v[1])]
    gate_up, dh = rnd(M, 2 * F), rnd(M, F)
    kept = bsmm.gated_act(gate_up)
    xi, wi = rnd(M, F, dtype=torch.float32), rnd(F, N, dtype=torch.float32)
    return {
        "quantize": lambda s: bsmm.quantize(p, (1, 32), "e4m3", "ue8m0", stream=s),
        "quantize_batch": lambda s: bsmm.quantize_batch([{"x": p, "block": (128, 128)}, {"x": w, "block": (1, 128)}],
                                                        stream=s),
        "quantize_atoms": lambda s: bsmm.quantize_atoms(p, stream=s),
        "gemm": lambda s: bsmm.gemm(pq, wq, ps, ws, stream=s),
        "gemm nvfp4": lambda s: bsmm.gemm(n4q, m4q, n4s, m4s, "e2m1", "e2m1", "ue4m3", stream=s),
        "gemm_atoms": lambda s: bsmm.gemm_atoms(pa[0], wa[0], pa[1], wa[1], stream=s),
        "gemm_grouped": lambda s: bsmm.gemm_grouped(gq, hq, gs, hs, stream=s),
        "int8_channel": lambda s: bsmm.int8_channel(xi, wi, return_acc=True, stream=s),
        "linear_backward": lambda s: bsmm.linear_backward(dyl, w, p, stream=s),
        "linear_backward_quantized": lambda s: bsmm.linear_backward_quantized(*ops, scales_are_atoms=True, stream=s),
        "linear_backward_checkpoint": lambda s: bsmm.linear_backward_checkpoint(dyl, w, pq, ps, stream=s),
        "gated_act": lambda s: bsmm.gated_act(gate_up, stream=s),
        "gated_act_backward": lambda s: bsmm.gated_act_backward(dh, kept[2], kept[3], return_h=True, stream=s),
        "adapters": lambda s: bsmm.adapters(x, a, b, ids, y=y, stream=s),
        "adapters_backward": lambda s: bsmm.adapters_backward(dy, x, a, b, ids, u, dx_base=x, stream=s),
    }


NAMES = ["quantize", "quantize_batch", "quantize_atoms", "gemm", "gemm nvfp4", "gemm_atoms", "gemm_grouped",
         "int8_channel", "linear_backward", "linear_backward_quantized", "linear_backward_checkpoint", "gated_act",
         "gated_act_backward", "adapters", "adapters_backward"]


@pytest.fixture(scope="module")
def made():
    c = calls()
    assert sorted(c) == sorted(NAMES)
    torch.cuda.synchronize()
    return c


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_from_the_streams_pool(made, name, monkeypatch):
    """Every tensor that the call allocates is allocated with `stream` current."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen, real = [], torch.empty

    def empty(*args, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*args, **kw)

    monkeypatch.setattr(torch, "empty", empty)
    made[name](s)
    monkeypatch.undo()
    s.synchronize()
    assert seen and all(v == s.cuda_stream for v in seen)


@pytest.mark.parametrize("name", NAMES)
def test_beside_late_work_of_the_current_stream(made, name):
    """Blocks that the host has freed but the current stream has yet to write:
    the call neither takes them nor waits for that work."""
    ref = [t.clone() for t in _tensors(made[name](None))]
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in ref] + [1 << 20, 1 << 22]
    s = torch.cuda.Stream()
    late = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    for t in late:
        t.fill_(0xFF)
    del late, t
    got = _tensors(made[name](s))
    s.synchronize()
    torch.cuda.synchronize()
    for p, q in zip(ref, got):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("name", ["adapters", "adapters_backward", "gated_act", "gated_act_backward",
                                  "linear_backward_checkpoint"])
def test_in_a_graph(made, name):
    """Captured with the launches' programmatic order, replayed three times."""
    ref = [t.clone() for t in _tensors(made[name](None))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _tensors(made[name](None))
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(ref, got):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_from_several_host_threads(made):
    """Each thread on a stream of its own, its calls back to back without a wait."""
    names = ["adapters", "adapters_backward", "gated_act", "gated_act_backward", "linear_backward_checkpoint"]
    ref = {n: [t.clone() for t in _tensors(made[n](None))] for n in names}
    torch.cuda.synchronize()
    errors = []

    def worker(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                got = [(n, _tensors(made[n](s))) for i in range(6) for n in names[k % 5:] + names[:k % 5]]
                s.synchronize()
                for n, ts in got:
                    for p, q in zip(ref[n], ts):
                        if not torch.equal(p.view(torch.uint8), q.view(torch.uint8)):
                            errors.append(f"thread {k}: {n} differs")
        except Exception as e:  # reported below, not lost in the thread
            errors.append(f"thread {k}: {e!r}")

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[:5]
    assert _bsmm().check_device_status()[0] == 0
