"""A block around an FP8 expert layer with gated activation: one training step and one decoding step.

    h = x + residual,  z = norm(h),  out = sum_j weight[j] W2[e] (act(A z) * (B z)),  W1[e] = [A; B]

for each token, e its chosen experts; h is the next block's residual. In training the norm and the gated
activation leave E4M3 codes in 1x128 groups for the products and their gradients E5M2 codes, and all gradients are
clipped to a largest norm; a decoding step is the norm, the router's product, the choice and the layer's two kernels.

    python examples/expert_block.py [--tokens 4096 --dim 4096 --hidden 2048 --experts 32 --top-k 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mx_block_scaled_amax_amd as qf8  # noqa: E402


def _blocks(w):
    """[experts][n][k] weights as codes and scales of 128x128 blocks."""
    parts = [qf8.quantize_block(e, 128, 128, qf8.E4M3, want_amax=False, pow2_scales=True)[:2] for e in w]
    return torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])


class ExpertBlock:
    """dim and hidden are multiples of 128. Weights are quantized once (after each update in training)."""

    def __init__(self, norm, router, w1, w2, top_k, act=qf8.ACT_SILU):
        self.norm, self.router, self.w1, self.w2 = norm, router, _blocks(w1), _blocks(w2)
        self.top_k, self.experts, self.act = top_k, w1.shape[0], act

    def _product(self, codes, weight, offsets, fmt, kind, rows=None):
        return qf8.matmul_block_experts(*codes, *weight, offsets, fmt, qf8.E4M3, kind, rows=rows, pow2_scales=True)

    def forward(self, x, residual):
        """x, residual [tokens][dim] BF16 -> out, h, and what backward() needs."""
        n = qf8.rms_norm_quantize(x, self.norm, qf8.E4M3, residual=residual, pow2_scales=True, want_y=True, want_rstd=True)
        logits = n.y @ self.router.t()
        ids, weights = qf8.route_experts(logits, self.top_k)
        offsets, rows, slots = qf8.order_experts(ids, self.experts, align=128)
        u = self._product((n.q, n.scales), self.w1, offsets, qf8.E4M3, qf8.WEIGHT_NK, rows=rows)
        a = qf8.gated_act_quantize(u, qf8.E4M3, act=self.act, pow2_scales=True)[:2]
        v = self._product(a, self.w2, offsets, qf8.E4M3, qf8.WEIGHT_NK)
        return qf8.combine_experts(v, weights, slots), n.h, (n, logits, ids, weights, offsets, rows, slots, u, a, v)

    def backward(self, dout, dh, saved):
        """From the gradients of out and of h: those of x (and of the residual), the norm, the router, w1 and w2."""
        n, logits, ids, weights, offsets, rows, slots, u, a, v = saved
        dv, dweights = qf8.combine_experts_backward(dout, v, weights, slots, rows)
        dv = qf8.quantize_block(dv, 1, 128, qf8.E5M2, want_amax=False, pow2_scales=True)[:2]
        dw2 = self._weight_gradient(dv, a, offsets)
        da = self._product(dv, self.w2, offsets, qf8.E5M2, qf8.WEIGHT_KN)
        du = qf8.gated_act_backward(da, u, qf8.E5M2, act=self.act, pow2_scales=True)[:2]
        held = (rows >= 0)[:, None]
        zr = (torch.where(held, n.q[rows.clamp(min=0).long()], 0), torch.where(held, n.scales[rows.clamp(min=0).long()], 1.0))
        dw1 = self._weight_gradient(du, zr, offsets)
        dz = qf8.combine_experts(self._product(du, self.w1, offsets, qf8.E5M2, qf8.WEIGHT_KN), torch.ones_like(weights), slots)
        dlogits = qf8.route_experts_backward(logits, ids, dweights)
        dx, dnorm = qf8.rms_norm_backward(dz + dlogits @ self.router, n.h, n.rstd, self.norm, dres=dh)
        return dx, dnorm, dlogits.t() @ n.y, dw1, dw2

    @staticmethod
    def _weight_gradient(dy, x, offsets):
        dyt = qf8.requantize_1x128_to_128x1(*dy, qf8.E5M2, qf8.E5M2)
        xt = qf8.requantize_1x128_to_128x1(*x, qf8.E4M3, qf8.E4M3)
        return qf8.matmul_block_experts_wgrad(*dyt, *xt, offsets, qf8.E5M2, qf8.E4M3, pow2_scales=True)

    def train(self, x, residual, dout, dh, max_norm):
        """One step: out, h, and the gradients, those of the weights clipped together to max_norm, with their norm."""
        out, h, saved = self.forward(x, residual)
        dx, *grads = self.backward(dout, dh, saved)
        return out, h, dx, grads, qf8.clip_grads(grads, max_norm)

    def decode(self, x, residual):
        """At most 64 tokens: out and h."""
        n = qf8.rms_norm_quantize(x, self.norm, None, residual=residual)
        ids, weights = qf8.route_experts(n.y @ self.router.t(), self.top_k)
        return qf8.expert_layer_tokens(n.y, *self.w1, *self.w2, ids, weights, qf8.E4M3, act=self.act), n.h


def reference(x, residual, norm, router, w1, w2, ids, act, dout, dh):
    """The block of these choices without quantization (fp32): out, h and the gradients of the first six by autograd."""
    leaves = [t.detach().float().requires_grad_() for t in (x, residual, norm, router, w1, w2)]
    xf, rf, nf, gf, a, b = leaves
    h = xf + rf
    z = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * nf
    chosen = (z @ gf.t()).softmax(1).gather(1, ids.long())
    weight = chosen / chosen.sum(1, keepdim=True)
    f = torch.nn.functional.silu if act == qf8.ACT_SILU else (lambda t: torch.nn.functional.gelu(t, approximate="tanh"))
    out = torch.zeros_like(xf)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            p, q = (z[t] @ a[e].t()).chunk(2, 1)
            out = out.index_add(0, t, weight[t, j][:, None] * ((f(p) * q) @ b[e].t()))
    torch.autograd.backward([out, h], [dout.float(), dh.float()])
    return (out.detach(), h.detach(), *(t.grad for t in leaves))


def inputs(tokens, dim, hidden, experts, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    return (normal(tokens, dim), normal(tokens, dim), 1 + 0.1 * normal(dim), normal(experts, dim) * dim ** -0.5,
            normal(experts, 2 * hidden, dim) * dim ** -0.5, normal(experts, dim, hidden) * hidden ** -0.5,
            normal(tokens, dim), normal(tokens, dim))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("dim", 4096), ("hidden", 2048), ("experts", 32), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    x, residual, norm, router, w1, w2, dout, dh = inputs(a.tokens, a.dim, a.hidden, a.experts)
    block = ExpertBlock(norm, router, w1, w2, a.top_k)

    def timed(f, n=10):
        f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(n):
            f()
        end.record()
        end.synchronize()
        return start.elapsed_time(end) / n * 1e3

    out, h, saved = block.forward(x, residual)
    got = (out, h, *block.backward(dout, dh, saved))
    want = reference(x, residual, norm, router, w1, w2, saved[2], block.act, dout, dh)
    for name, g, w in zip(("out", "h", "dx", "dnorm", "drouter", "dw1", "dw2"), got, (*want[:3], *want[4:])):
        print(f"{name}: relative difference from the block without quantization {float((g.float() - w).norm() / w.norm()):.3f}")
    print(f"training step, {a.tokens} tokens: {timed(lambda: block.train(x, residual, dout, dh, 1.0)):.0f} us")
    few, res = x[:64].contiguous(), residual[:64].contiguous()
    print(f"decoding step, {few.shape[0]} tokens: {timed(lambda: block.decode(few, res)):.0f} us")


if __name__ == "__main__":
    main()
