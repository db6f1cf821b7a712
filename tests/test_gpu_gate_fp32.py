"""The gated activation's FP32 results over the whole range of gates, each value for itself.

Tolerances. exp2 is an ulp off (2^-23), its argument's rest 2^-24, 1 + e a half step that counts for less than e, the reciprocal an ulp:
s within 2^-21.2 of itself, and so 1 - s = e s with two roundings more. act(a) b has two more, 2^-24 each: 2^-20. The slope's terms s
and a s (1 - s) z': at most 2^-20.2 and six roundings of 2^-24 of them, 2^-19. Where the sigmoid falls below 2^-126 it may be 0: off by 2^-126 times 1 + |a| z' in the slope, which is 89 for SiLU
(a = -88) and, for GELU, whose z is -87.4 at a = -10, 1 + 10 x 1.596 (1 + 0.1342 x 100) = 231: below 2^-118."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_gate import ACTS, TINY, parts

pytestmark = pytest.mark.gpu


def gates():
    gen = torch.Generator(device="cuda").manual_seed(11)
    near = torch.linspace(-14, 14, 128 * 512, device="cuda")
    far = torch.linspace(-100, 100, 128 * 64, device="cuda")
    small = torch.randn(128 * 64, generator=gen, device="cuda") * 2.0 ** (-20 * torch.rand(128 * 64, generator=gen, device="cuda"))
    a = torch.cat([near, far, small]).view(-1, 128)
    return a, 1 + torch.rand(a.shape, generator=gen, device="cuda"), torch.randn(a.shape, generator=gen, device="cuda")


@pytest.mark.parametrize("act", ACTS)
def test_values(act):
    a, b, _ = gates()
    y = qf8.gated_act_quantize(torch.cat([a, b], 1), None, act=act)[2].double()
    want = parts(act, a.double())[0] * b.double()
    off = (y - want).abs() - TINY * b.double()
    assert float((off / want.abs().clamp(min=2.0 ** -126)).max()) <= 2.0 ** -20


@pytest.mark.parametrize("act", ACTS)
def test_gradients(act):
    a, b, dy = gates()
    dx = qf8.gated_act_backward(dy, torch.cat([a, b], 1), None, act=act)[2].double()
    y, slope = parts(act, a.double())
    s = torch.where(a == 0, 0.5, y / a.double())
    terms = s + (slope - s).abs()
    want = torch.cat([dy.double() * b.double() * slope, dy.double() * y], 1)
    size = torch.cat([(dy.double() * b.double()).abs() * terms * 2.0 ** -19, want[:, 128:].abs() * 2.0 ** -20], 1)
    assert bool(((dx - want).abs() <= size + torch.cat([2 * TINY * (dy * b).abs(), TINY * dy.abs()], 1)).all())
