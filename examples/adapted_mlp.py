"""A gated MLP whose frozen-precision projections are MXFP8 and whose requests
bring low-rank adapters: a training step from 8-bit checkpoints, and a decode
step.

    python examples/adapted_mlp.py [--tokens T] [--dim D] [--inner I] [--rank R] [--adapters L]

    y = (act(gate) * up) W2^T,  [gate | up] = x W1^T + s[id] (x A[id]^T) B[id]^T

Training keeps x and gate_up in 8 bits (x's codes and scales are those of the
forward's MXFP8 operand; gate_up's come out of the gated activation's one pass)
and h as the codes that the second projection read anyway.  The backward pass
takes all of its gradients from them.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_gemm_gb300 as bsmm  # noqa: E402


class AdaptedMlp:
    """Weights W1 [2 I, D], W2 [D, I] and adapters a [L, R, D], b [L, 2 I, R],
    all bfloat16; the projections' MXFP8 operands are made once."""

    def __init__(self, w1, w2, a, b, scaling, act="silu"):
        self.w1, self.w2, self.a, self.b, self.scaling, self.act = w1, w2, a, b, scaling, act
        self.q1 = bsmm.quantize(w1, (1, 32), "e4m3", "ue8m0")
        self.q2 = bsmm.quantize(w2, (1, 32), "e4m3", "ue8m0")
        self.q2_atoms = bsmm.quantize_atoms(w2)

    def _project(self, codes, scales, q):
        return bsmm.gemm(codes, q[0], scales, q[1], out_dtype=torch.bfloat16)[0]

    def forward(self, x, ids):
        """``(y, saved)`` of x [T, D] bfloat16, ids [T] int32."""
        xq, xs = bsmm.quantize(x, (1, 32), "e4m3", "ue8m0")
        gate_up = self._project(xq, xs, self.q1)
        _, u = bsmm.adapters(x, self.a, self.b, ids, y=gate_up, scaling=self.scaling, out=gate_up)
        h, hs, codes, scales = bsmm.gated_act(gate_up, act=self.act, code="int8", scale="f32")
        y = self._project(h, hs, self.q2)
        return y, (xq, xs, u, ids, codes, scales, h, hs)

    def backward(self, dy, saved):
        """Gradients of x, W1, W2, a and b from dy [T, D] bfloat16."""
        xq, xs, u, ids, codes, scales, h, hs = saved
        dh, dw2 = bsmm.linear_backward_checkpoint(dy, self.w2, h, hs)
        d_gate_up, _ = bsmm.gated_act_backward(dh, codes, scales, act=self.act, code="int8", scale="f32")
        dx, dw1 = bsmm.linear_backward_checkpoint(d_gate_up, self.w1, xq, xs)
        dx, da, db = bsmm.adapters_backward(d_gate_up, xq, self.a, self.b, ids, u, scaling=self.scaling, dx_base=dx,
                                            x_scales=xs, dx=dx)
        return dx, dw1, dw2, da, db

    def decode(self, x, ids):
        """y of a few tokens, keeping nothing: h's scales go straight into the
        layout that the second projection reads."""
        xq, xs = bsmm.quantize(x, (1, 32), "e4m3", "ue8m0")
        gate_up = self._project(xq, xs, self.q1)
        bsmm.adapters(x, self.a, self.b, ids, y=gate_up, scaling=self.scaling, out=gate_up)
        h, hs, _, _ = bsmm.gated_act(gate_up, act=self.act, code=None, h_scales_are_atoms=True)
        T, (D, I) = x.shape[0], self.w2.shape
        return bsmm.gemm_atoms(h.view(1, T, I), self.q2_atoms[0].view(1, D, I), hs, self.q2_atoms[1],
                               out_dtype=torch.bfloat16)[0]


def make(dim, inner, rank, adapters, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(device=device, dtype=torch.bfloat16)

    return AdaptedMlp(t(2 * inner, dim, scale=dim ** -0.5), t(dim, inner, scale=inner ** -0.5),
                      t(adapters, rank, dim, scale=dim ** -0.5), t(adapters, 2 * inner, rank, scale=rank ** -0.5),
                      torch.linspace(0.5, 1.5, adapters, device=device))


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--dim", type=int, default=4096)
    p.add_argument("--inner", type=int, default=8192)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--adapters", type=int, default=8)
    args = p.parse_args()
    mlp = make(args.dim, args.inner, args.rank, args.adapters)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(args.tokens, args.dim, device="cuda", generator=g).bfloat16()
    dy = torch.randn(args.tokens, args.dim, device="cuda", generator=g).bfloat16()
    ids = torch.randint(0, args.adapters, (args.tokens,), device="cuda", dtype=torch.int32, generator=g)

    def timed(f, n=20):
        for _ in range(3):
            r = f()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        e0.record()
        for _ in range(n):
            r = f()
        e1.record()
        torch.cuda.synchronize()
        return r, e0.elapsed_time(e1) / n * 1e3

    (y, saved), fwd = timed(lambda: mlp.forward(x, ids))
    grads, bwd = timed(lambda: mlp.backward(dy, saved))
    small, dec = timed(lambda: mlp.decode(x[:64], ids[:64]))
    kept = sum(t.numel() * t.element_size() for t in saved)
    print(f"forward {fwd:.1f} us, backward {bwd:.1f} us, decode of 64 tokens {dec:.1f} us")
    print(f"kept for the backward pass: {kept / 1e6:.1f} MB")
    print("decode against forward:", float((small.float() - y[:64].float()).norm() / y[:64].float().norm()))


if __name__ == "__main__":
    main()
