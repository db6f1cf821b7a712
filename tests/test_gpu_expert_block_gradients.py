"""The gradients of examples/expert_block.py, each against the block without quantization in 64 bits.

Tolerances, relative to the norm. A rounding to E4M3 is off by at most half a step, 2^-4, of the power of two below a value: evenly spread,
r = 2^-4 / sqrt(3) = 0.036 of the norm at most; E5M2 2 r, which counts as 4 in squares. Independent ones add in squares:
  out   z and w1 in each half of the gate, the activation, w2: 6
  dw2   dv twice (E5M2, re-grouped): 8; the activation twice and what it holds of z and w1: 6
  dw1   du twice: 8; what it holds of dv 4, w2 1, z and w1 in the two halves 4; z twice: 2
  dz    du once: 4, w1 1, and what du holds: 9; with it dnorm, and dx but for dh, which is added to it unrounded
  drouter   that of out; the choice's gradient is a difference of such products: twice that
Roundings to BF16 (2^-9 / sqrt(3) of the norm) are below a tenth of r."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_expert_block import example
from test_gpu_gate import parts

pytestmark = pytest.mark.gpu
R = 2.0 ** -4 / math.sqrt(3)


class Act(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, act):
        y, slope = parts(act, a)
        ctx.save_for_backward(slope)
        return y

    @staticmethod
    def backward(ctx, dy):
        return dy * ctx.saved_tensors[0], None


def exact(x, residual, norm, router, w1, w2, ids, act, dout, dh, choice=True):
    """out and the gradients of x, norm, router, w1, w2; choice: with the path through the choice's weights."""
    leaves = [t.detach().double().requires_grad_() for t in (x, norm, router, w1, w2)]
    xd, nd, gd, a, b = leaves
    h = xd + residual.double()
    z = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * nd
    weight = (z if choice else z.detach()) @ gd.t()
    weight = weight.softmax(1).gather(1, ids.long())
    weight = weight / weight.sum(1, keepdim=True)
    out = torch.zeros_like(xd)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            p, q = (z[t] @ a[e].t()).chunk(2, 1)
            out = out.index_add(0, t, weight[t, j][:, None] * ((Act.apply(p, act) * q) @ b[e].t()))
    torch.autograd.backward([out, h], [dout.double(), dh.double()])
    return [out.detach()] + [t.grad for t in leaves]


def off(got, want):
    assert got.shape == want.shape and bool(torch.isfinite(got).all())
    return float((got.double() - want.double()).norm()) / float(want.double().norm())


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k,act", [
    (300, 512, 256, 8, 2, qf8.ACT_SILU), (130, 384, 128, 16, 4, qf8.ACT_GELU), (520, 256, 384, 4, 3, qf8.ACT_GELU), (200, 640, 256, 6, 1, qf8.ACT_SILU)])
def test_each_gradient(tokens, dim, hidden, experts, top_k, act):
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(tokens, dim, hidden, experts, seed=tokens)
    block = example.ExpertBlock(norm, router, w1, w2, top_k, act=act)
    out, h, saved = block.forward(x, residual)
    dx, dnorm, drouter, dw1, dw2 = block.backward(dout, dh, saved)
    want = exact(x, residual, norm, router, w1, w2, saved[2], act, dout, dh)
    assert off(out, want[0]) <= math.sqrt(6) * R
    assert off(dw2, want[5]) <= math.sqrt(14) * R
    assert off(dw1, want[4]) <= math.sqrt(19) * R
    assert off(dnorm, want[2]) <= math.sqrt(14) * R
    rounding = 2.0 ** -8 * float(want[1].norm() / (want[1] - dh.double()).norm())
    assert off(dx.double() - dh.double(), want[1] - dh.double()) <= math.sqrt(14) * R + rounding
    if top_k > 1:
        assert off(drouter, want[3]) <= math.sqrt(12) * R
    else:                                                     # one weight, which is 1: no gradient but roundings of 2^-24 of <dout, v>
        v = saved[9].double().norm(dim=1).max()
        assert float(drouter.double().norm()) <= 2.0 ** -20 * float(dout.double().norm() * v * saved[0].y.double().norm())


def test_the_choice_reaches_the_input():
    """What the router adds to dx by itself: the difference of two backward passes, with the router and with zeros in its place, and no dh. Each
    pass rounds dz and dx to BF16 a few times, 2^-8 of dx in all; beside them the choice's gradient, as drouter's."""
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(400, 512, 256, 8, seed=17)
    router, dh = 4 * router, torch.zeros_like(dh)
    block = example.ExpertBlock(norm, router, w1, w2, 3)
    _, _, saved = block.forward(x, residual)
    every = block.backward(dout, dh, saved)[0].double()
    block.router = torch.zeros_like(router)
    none = block.backward(dout, dh, saved)[0].double()
    args = (x, residual, norm, router, w1, w2, saved[2], qf8.ACT_SILU, dout, dh)
    want, without = exact(*args)[1], exact(*args, choice=False)[1]
    part = want - without
    assert off(none, without) <= math.sqrt(14) * R
    assert off(every - none, part) <= math.sqrt(12) * R + 2 * 2.0 ** -8 * float(want.norm() / part.norm())
