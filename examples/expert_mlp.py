"""A mixture of gated MLPs in MXFP8: a training step with its AdamW update, and a
decode step.

    python examples/expert_mlp.py [--tokens T] [--dim D] [--inner I] [--experts E] [--top K]

    y[t] = sum over the k experts e of token t of  p[t, e] (act(gate) * up) W2[e]^T,
    [gate | up] = x[t] W1[e]^T,  p the softmax of the router's chosen logits x Wr^T

No size of an expert's share is known on the host: the offsets stay on the GPU,
so that a step can be captured into a graph as it stands.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_gemm_gb300 as bsmm  # noqa: E402


class ExpertMlp:
    """Binary32 weights wr [E, D], w1 [E, 2 I, D], w2 [E, D, I] with their
    bfloat16 copies, 8-bit AdamW states and the forward's MXFP8 operands."""

    def __init__(self, wr, w1, w2, top, act="silu"):
        self.masters = [wr.float(), w1.float(), w2.float()]
        self.copies = [w.bfloat16() for w in self.masters]
        self.top, self.act, self.steps = top, act, 0
        n = [w.numel() for w in self.masters]
        self.m, self.v = ([torch.zeros_like(w, dtype=torch.uint8) for w in self.masters] for _ in range(2))
        self.m_scales, self.v_scales = ([torch.zeros((k + 127) // 128, device=wr.device) for k in n] for _ in range(2))
        self._operands()

    def _operands(self):
        self.q = []
        for w in self.copies[1:]:
            E, N, K = w.shape
            codes, atoms = bsmm.quantize_atoms(w.view(E * N, K), batches=E)
            self.q.append((codes.view(E, N, K), atoms))

    def forward(self, x, keep=True):
        """``(y, saved)`` of x [T, D] bfloat16; without ``keep`` nothing is saved."""
        logits = x @ self.copies[0].t()
        weights, ids, offsets, rows, slots = bsmm.route(logits, self.top)
        xq, xs = bsmm.quantize(x, (1, 32), "e4m3", "ue8m0")
        gate_up = bsmm.expert_gemm(xq, xs, *self.q[0], offsets, rows=rows)
        h, hs, codes, scales = bsmm.gated_act(gate_up, act=self.act, code="int8" if keep else None)
        down = bsmm.expert_gemm(h, hs, *self.q[1], offsets)
        y = bsmm.expert_combine(down, slots, weights)
        return y, ((x, logits, weights, ids, offsets, rows, slots, codes, scales, down) if keep else None)

    def backward(self, dy, saved):
        """Gradients of x, wr, w1 and w2 from dy [T, D] bfloat16."""
        x, logits, weights, ids, offsets, rows, slots, codes, scales, down = saved
        d_down, d_weights = bsmm.expert_combine_backward(dy, down, slots, weights)
        dh_shape = (down.shape[0], self.copies[2].shape[2])
        h = bsmm.gated_act_backward(torch.zeros(dh_shape, device=dy.device, dtype=torch.bfloat16), codes, scales,
                                    act=self.act, return_h=True)[1]
        dh, dw2 = bsmm.expert_backward(d_down, self.copies[2], h, offsets)
        d_gate_up, _ = bsmm.gated_act_backward(dh, codes, scales, act=self.act)
        dx, dw1 = bsmm.expert_backward(d_gate_up, self.copies[1], x, offsets, rows=rows)
        d_logits = bsmm.route_backward(d_weights, logits, ids, weights)
        dx = bsmm.expert_combine(dx, slots, out_dtype=torch.float32) + (d_logits @ self.copies[0]).float()
        return dx.bfloat16(), d_logits.t() @ x, dw1, dw2

    def update(self, grads, lr=1e-3):
        """One AdamW step; the forward's operands follow the new weights."""
        self.steps += 1
        bsmm.adamw(self.masters, grads, self.m, self.v, self.steps, lr=lr, m_scales=self.m_scales, v_scales=self.v_scales,
                   copies=self.copies)
        self._operands()


def make(dim, inner, experts, top, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def t(*shape, scale):
        return (torch.randn(*shape, generator=g) * scale).to(device)

    return ExpertMlp(t(experts, dim, scale=dim ** -0.5), t(experts, 2 * inner, dim, scale=dim ** -0.5),
                     t(experts, dim, inner, scale=inner ** -0.5), top)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=8192)
    p.add_argument("--dim", type=int, default=2048)
    p.add_argument("--inner", type=int, default=2048)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--top", type=int, default=2)
    args = p.parse_args()
    mlp = make(args.dim, args.inner, args.experts, args.top)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(args.tokens, args.dim, device="cuda", generator=g).bfloat16() for _ in range(2))

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

    (_, saved), fwd = timed(lambda: mlp.forward(x))
    grads, bwd = timed(lambda: mlp.backward(dy, saved))
    _, upd = timed(lambda: mlp.update(grads[1:]))
    _, dec = timed(lambda: mlp.forward(x[:8], keep=False))
    print(f"forward {fwd:.1f} us, backward {bwd:.1f} us, update {upd:.1f} us, decode of 8 tokens {dec:.1f} us")


if __name__ == "__main__":
    main()
