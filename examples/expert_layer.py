"""A mixture-of-experts layer in FP8: one training step and one decoding step.

    y[t] = sum_j weight[t][j] * W2[e] silu(W1[e] x[t]),   e = ids[t][j]

Activations and gradients are quantized in 1x128 groups (E4M3 forward, E5M2 backward), weights in
128x128 blocks, all with power-of-two scales; every product takes the codes. torch does the router's
product and the activation.

    python examples/expert_layer.py [--tokens 4096 --dim 4096 --hidden 2048 --experts 32 --top-k 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mx_block_scaled_amax_amd as qf8  # noqa: E402


def _groups(x, fmt):
    """Codes and scales in 1x128 groups."""
    return qf8.quantize_block(x, 1, 128, fmt, want_amax=False, pow2_scales=True)[:2]


def _blocks(w):
    """[experts][n][k] weights as codes and scales of 128x128 blocks."""
    parts = [qf8.quantize_block(e, 128, 128, qf8.E4M3, want_amax=False, pow2_scales=True)[:2] for e in w]
    return torch.stack([q for q, _ in parts]), torch.stack([s for _, s in parts])


class ExpertLayer:
    """Sizes are multiples of 16, as the quantizer needs them. Weights are quantized once (after each update
    in training)."""

    def __init__(self, router, w1, w2, top_k, score=qf8.SCORE_SOFTMAX, bias=None, groups=1, top_groups=1, scale=1.0):
        self.router, self.w1, self.w2 = router, _blocks(w1), _blocks(w2)
        self.top_k, self.experts = top_k, w1.shape[0]
        self.gate = dict(score=score, renorm=True, scale=scale)
        self.choice = dict(bias=bias, groups=groups, top_groups=top_groups)

    def _product(self, codes, weight, offsets, fmt, kind, rows=None):
        return qf8.matmul_block_experts(*codes, *weight, offsets, fmt, qf8.E4M3, kind, rows=rows, pow2_scales=True)

    def forward(self, x, training=False):
        """x [tokens][dim] BF16 -> y, and what backward() needs. In training every expert's rows start at a
        multiple of 128, the groups of the weight gradients."""
        logits = x @ self.router.t()
        ids, weights = qf8.route_experts(logits, self.top_k, **self.gate, **self.choice)
        offsets, rows, slots = qf8.order_experts(ids, self.experts, align=128 if training else 1)
        u = self._product(_groups(x, qf8.E4M3), self.w1, offsets, qf8.E4M3, qf8.WEIGHT_NK, rows=rows)
        act = _groups(torch.nn.functional.silu(u), qf8.E4M3)
        v = self._product(act, self.w2, offsets, qf8.E4M3, qf8.WEIGHT_NK)
        y = qf8.combine_experts(v, weights, slots)
        return y, (x, logits, ids, weights, offsets, rows, slots, u, act, v)

    def backward(self, dy, saved):
        """Gradients of x, the router, w1 and w2 (the weights' in FP32)."""
        x, logits, ids, weights, offsets, rows, slots, u, act, v = saved
        dv, dweights = qf8.combine_experts_backward(dy, v, weights, slots, rows)
        dv = _groups(dv, qf8.E5M2)
        dw2 = self._weight_gradient(dv, act, offsets)
        dact = self._product(dv, self.w2, offsets, qf8.E5M2, qf8.WEIGHT_KN)
        sig = torch.sigmoid(u.float())
        du = _groups((dact.float() * (sig * (1 + u.float() * (1 - sig)))).to(torch.bfloat16), qf8.E5M2)
        xr = _groups(torch.where((rows >= 0)[:, None], x[rows.clamp(min=0).long()], 0), qf8.E4M3)
        dw1 = self._weight_gradient(du, xr, offsets)
        dx = self._product(du, self.w1, offsets, qf8.E5M2, qf8.WEIGHT_KN)
        dx = qf8.combine_experts(dx, torch.ones_like(weights), slots)
        dlogits = qf8.route_experts_backward(logits, ids, dweights, **self.gate)
        return dx + dlogits @ self.router, dlogits.t() @ x, dw1, dw2

    @staticmethod
    def _weight_gradient(dy, x, offsets):
        dyt = qf8.requantize_1x128_to_128x1(*dy, qf8.E5M2, qf8.E5M2)
        xt = qf8.requantize_1x128_to_128x1(*x, qf8.E4M3, qf8.E4M3)
        return qf8.matmul_block_experts_wgrad(*dyt, *xt, offsets, qf8.E5M2, qf8.E4M3, pow2_scales=True)


def reference(x, router, w1, w2, ids, dy, scale=1.0):
    """The layer of these choices without quantization (fp32), and its gradients by autograd."""
    leaves = [t.detach().float().requires_grad_() for t in (x, router, w1, w2)]
    xf, rf, a, b = leaves
    chosen = (xf @ rf.t()).softmax(1).gather(1, ids.long())
    gate = scale * chosen / chosen.sum(1, keepdim=True)
    y = torch.zeros_like(xf)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            out = torch.nn.functional.silu(xf[t] @ a[e].t()) @ b[e].t()
            y = y.index_add(0, t, gate[t, j][:, None] * out)
    y.backward(dy.float())
    return (y.detach(), *(t.grad for t in leaves))


def inputs(tokens, dim, hidden, experts, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    return (normal(tokens, dim), normal(experts, dim) * dim ** -0.5, normal(experts, hidden, dim) * dim ** -0.5,
            normal(experts, dim, hidden) * hidden ** -0.5, normal(tokens, dim))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("dim", 4096), ("hidden", 2048), ("experts", 32), ("top-k", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    x, router, w1, w2, dy = inputs(a.tokens, a.dim, a.hidden, a.experts)
    layer = ExpertLayer(router, w1, w2, a.top_k)

    def timed(f, n=10):
        f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(n):
            f()
        end.record()
        end.synchronize()
        return start.elapsed_time(end) / n * 1e3

    y, saved = layer.forward(x, training=True)
    got = (y, *layer.backward(dy, saved))
    want = reference(x, router, w1, w2, saved[2], dy)
    for name, g, w in zip(("y", "dx", "drouter", "dw1", "dw2"), got, want):
        print(f"{name}: relative difference from the layer without quantization {float((g.float() - w).norm() / w.norm()):.3f}")
    print(f"training step, {a.tokens} tokens: {timed(lambda: layer.backward(dy, layer.forward(x, training=True)[1])):.0f} us")
    few = x[:64].contiguous()
    print(f"decoding step, {few.shape[0]} tokens: {timed(lambda: layer.forward(few)):.0f} us")


if __name__ == "__main__":
    main()
