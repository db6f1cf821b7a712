"""The choice of experts at the ends of the range: infinities and largest values, chosen experts whose
scores underflow, experts that bias or mask shut out."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_experts import HALF, SCORE, check_route, random_logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [1, 9000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinity_is_the_largest_value_of_its_type(dtype, tokens, score):
    """+Inf ties with the type's largest value, in the order and in the weights."""
    x = torch.zeros(tokens, 16, dtype=dtype, device="cuda")
    x[:, 9] = math.inf
    x[:, 3] = torch.finfo(dtype).max
    for bias in (None, torch.zeros(16, device="cuda")):
        ids, w = qf8.route_experts(x, 2, score=SCORE[score], bias=bias)
        assert bool((ids == torch.tensor([3, 9], device="cuda")).all())
        assert bool((w == 0.5).all()), w[0].tolist()
        dw = torch.tensor([[1.0, 0.0]], device="cuda").expand(tokens, 2).contiguous()
        d = qf8.route_experts_backward(x, ids, dw, score=SCORE[score]).float()
        want = torch.zeros(16, device="cuda")
        if score == "softmax":                               # p (g - mean) with p = 1/2 each; a sigmoid is flat there
            want[3], want[9] = 0.25, -0.25
        assert bool((d == want).all()), d[0].tolist()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-800.0, -30000.0, None])
def test_weights_of_chosen_experts_whose_scores_underflow(dtype, low):
    """The bias chooses experts far below the largest logit: softmax scores that underflow have ratios all the
    same, and the gradient is that of the weights."""
    low = torch.finfo(dtype).min / 2 if low is None else low
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.randn(40, 24, generator=gen, device="cuda")
    x[:, 12:] = low if abs(low) > 1e6 else low + 2.0 * x[:, 12:]
    x = x.to(dtype)
    bias = torch.zeros(24, device="cuda")
    bias[14:19] = torch.linspace(3.0, 2.0, 5, device="cuda")
    ids, w = qf8.route_experts(x, 4, bias=bias, scale=1.5)
    assert bool((ids == torch.arange(14, 18, device="cuda")).all())
    l = x.double().cpu().requires_grad_()
    chosen = l.gather(1, ids.long().cpu())
    want = 1.5 * torch.softmax(chosen, 1)
    assert bool(((w.double().cpu() - want).abs() <= want * (2.0 ** -24 * 1.01) + 1e-45).all()), w[0].tolist()
    dw = torch.randn(40, 4, generator=gen, device="cuda")
    got = qf8.route_experts_backward(x, ids, dw, scale=1.5).double().cpu()
    (grad,) = torch.autograd.grad(want, l, dw.double().cpu())
    tol = grad.abs() * HALF[dtype] * 1.01 + 2.0 ** -45 * dw.abs().double().cpu().max(dim=1, keepdim=True)[0]
    assert bool(((got - grad).abs() <= tol).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_choice_is_score_plus_bias_in_masked_places(score, dtype):
    """With a bias or groups a masked logit is compared by 0 + bias, as the formula has it; its weight is 0. A
    bias of -Inf shuts an expert out."""
    x, _ = random_logits(50, 64, dtype, 77)
    x[:, 5] = -math.inf
    x[:, 20] = math.nan
    x[3, 8:] = -math.inf
    x[4] = -math.inf
    bias = torch.linspace(-0.2, 0.2, 64, device="cuda")
    bias[5] = 5.0
    ids, w = check_route(x, 6, score, bias=bias)
    assert bool((ids[:, 0] == 5).all()) and bool((w[:, 0] == 0).all())
    check_route(x, 6, score, bias=bias, groups=8, top_groups=3)
    check_route(x, 6, score, groups=8, top_groups=3)
    bias[[2, 5, 17, 40]] = -math.inf
    ids, w = check_route(x, 6, score, bias=bias)
    assert not bool(((ids == 2) | (ids == 5) | (ids == 17) | (ids == 40)).any())
    ids, w = check_route(x, 6, score, bias=bias, groups=8, top_groups=3)
    assert not bool(((ids == 2) | (ids == 5) | (ids == 17) | (ids == 40)).any())


@pytest.mark.parametrize("tokens", [3, 3000])
def test_lowest_value_is_a_number(tokens):
    """Without bias and groups -Inf comes after the type's lowest value, at a higher index too."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((tokens, 96), -math.inf, dtype=dtype, device="cuda")
        x[:, 50:53] = torch.finfo(dtype).min
        x[:, 70] = 0.0
        for score in ("softmax", "sigmoid"):
            ids, _ = check_route(x, 5, score)
            assert ids[tokens - 1].tolist() == [70, 50, 51, 52, 0]


@pytest.mark.parametrize("tokens", [5, 3000])
@pytest.mark.parametrize("at", [-600.0, -700.0, -708.0])
def test_gradient_of_small_sigmoid_scores(tokens, at):
    """Scores near fp64's smallest have ratios, and a gradient, like others: there a sigmoid is exp, so the
    renormalised weights are a softmax of the chosen logits and 1 - p is 1."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    x = at + torch.rand(tokens, 20, generator=gen, device="cuda")
    ids, w = qf8.route_experts(x, 4, score=qf8.SCORE_SIGMOID)
    chosen = torch.softmax(x.double().gather(1, ids.long()), 1)
    # fp64's own error: 2^-52 of an exponent of up to 709, doubled for the sum
    slack = 2.0 ** -24 * 1.01 + 2.0 ** -40
    assert bool(((w.double() - chosen).abs() <= chosen * slack).all())
    dw = 30.0 * torch.randn(tokens, 4, generator=gen, device="cuda")
    got = qf8.route_experts_backward(x, ids, dw, score=qf8.SCORE_SIGMOID).double()
    g = dw.double()
    want = torch.zeros_like(got).scatter_(1, ids.long(), chosen * (g - (g * chosen).sum(1, keepdim=True)))
    assert bool(((got - want).abs() <= want.abs() * slack + 2.0 ** -40 * g.abs().max(1, keepdim=True)[0]).all())
