"""bsmm_adamw's in-place changes as autograd sees them."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _bsmm():
    import block_scaled_precision_gemm_gb300 as bsmm
    return bsmm


def zeros(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype, device="cuda")


@pytest.mark.parametrize("bits8", [False, True])
def test_versions_of_what_is_written_rise(bits8):
    """Those of the parameters and their copies; the gradients' and the schedule's stay."""
    bsmm = _bsmm()
    n = 300
    p = [torch.nn.Parameter(zeros(n)), zeros(n)]
    g = [torch.ones(n, device="cuda") for _ in p]
    m, v = ([zeros(n, torch.uint8 if bits8 else torch.float32) for _ in p] for _ in range(2))
    scales = {k: [zeros(3) for _ in p] for k in ("m_scales", "v_scales")} if bits8 else {}
    copies, hyper = [zeros(n, torch.bfloat16) for _ in p], torch.tensor([0.1, 1.0, 1.0], device="cuda")
    written = [*p, *copies]
    read = [*g, hyper]
    before = [t._version for t in written], [t._version for t in read]
    bsmm.adamw(iter(p), tuple(g), iter(m), iter(v), 1, lr=0.1, copies=iter(copies), hyper=hyper, **scales)
    assert all(t._version > a for t, a in zip(written, before[0])) and [t._version for t in read] == before[1]


@pytest.mark.parametrize("which", ["parameter", "copy"])
def test_a_backward_pass_over_a_step_raises(which):
    bsmm = _bsmm()
    w = torch.nn.Parameter(torch.randn(8, 8, device="cuda"))
    copy = w.detach().bfloat16()
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    y = x @ w if which == "parameter" else x.bfloat16() @ copy
    bsmm.adamw([w], [torch.ones_like(w)], [torch.zeros_like(w)], [torch.zeros_like(w)], 1, lr=0.1, copies=[copy])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_tensors_made_in_inference_mode():
    """They have no versions, and are updated all the same."""
    with torch.inference_mode():
        p, g, m, v = torch.ones(5, device="cuda"), torch.ones(5, device="cuda"), zeros(5), zeros(5)
    _bsmm().adamw([p], [g], [m], [v], 1, lr=0.5, weight_decay=0.0)
    assert torch.equal(p.cpu(), torch.full((5,), 0.5))
