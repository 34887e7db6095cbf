"""The example's adapted MLP, forward, backward and decode, against autograd in
float64 on unquantized operands.

Tolerances.  E4M3 keeps 3 mantissa bits: a value's relative error is uniform up
to 2^-4, 0.026 root mean square over a binade, and independent from element to
element, so a contraction of two quantized operands is off by 0.026 sqrt(2) =
0.037 of its norm; E5M2 (2 bits) doubles its operand's share: sqrt(0.026^2 +
0.052^2) = 0.058.  A gradient passes at most two such backward products and the
forward's three quantized activations (x, gate_up's INT8, h): sqrt(2 * 0.058^2 +
2 * 0.037^2 + 0.01^2) = 0.1, taken twice for the nonlinearity: 0.2.  The output
passes two forward products: sqrt(2) * 0.037 = 0.053, taken twice: 0.11."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("adapted_mlp", os.path.join(ROOT, "examples", "adapted_mlp.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,rank,adapters", [(96, 8, 3), (640, 16, 5), (2048, 32, 2)])
def test_step_against_autograd(tokens, rank, adapters):
    import block_scaled_precision_gemm_gb300 as bsmm
    mlp = _example().make(512, 768, rank, adapters, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, 512, device="cuda", generator=g).bfloat16()
    dy = torch.randn(tokens, 512, device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, adapters, (tokens,), device="cuda", dtype=torch.int32, generator=g)
    y, saved = mlp.forward(x, ids)
    got = mlp.backward(dy, saved)

    leaves = [t.double().requires_grad_() for t in (x, mlp.w1, mlp.w2, mlp.a, mlp.b)]
    lx, w1, w2, a, b = leaves
    at = ids.clamp(min=0).long()
    s = torch.where(ids >= 0, mlp.scaling.double()[at], torch.zeros((), device="cuda", dtype=torch.float64))
    low = torch.einsum("trd,td->tr", a[at], lx)
    gate_up = lx @ w1.T + s[:, None] * torch.einsum("tnr,tr->tn", b[at], low)
    gate, up = gate_up.chunk(2, dim=1)
    want = (torch.nn.functional.silu(gate) * up) @ w2.T
    want.backward(dy.double())
    assert _rel(y, want.detach()) < 0.11
    for name, g1, leaf in zip(("dx", "dw1", "dw2", "da", "db"), got, leaves):
        assert _rel(g1, leaf.grad) < 0.2, name

    few = mlp.decode(x[:7], ids[:7])
    assert _rel(few, want.detach()[:7]) < 0.11
    assert bsmm.check_device_status()[0] == 0
