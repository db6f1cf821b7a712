"""The expert layer's operators at the sizes where another kernel or launch shape takes over, on both sides."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_experts import HALF, check_route, combine_case, plain_order, random_logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("choices", [2047, 2048, 2049, 3071, 4095, 4096, 4097])
@pytest.mark.parametrize("align", [1, 16])
def test_order(choices, align):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(choices)
    ids = torch.randint(-1, 41, (choices, 1), generator=gen, device="cuda", dtype=torch.int32)
    offsets, rows, slots = qf8.order_experts(ids, 40, align=align)
    want = plain_order(ids.cpu(), 40, align, rows.numel())
    assert offsets.tolist() == want[0] and rows.tolist() == want[1] and slots.reshape(-1).tolist() == want[2]


@pytest.mark.parametrize("tokens", [1023, 1024, 1025, 2047, 2048, 2049])
def test_route(tokens):
    for dtype in (torch.bfloat16, torch.float32):
        x, gen = random_logits(tokens, 72, dtype, tokens)
        bias = 0.1 * torch.randn(72, generator=gen, device="cuda")
        check_route(x, 5)
        check_route(x, 5, "sigmoid", bias=bias, groups=8, top_groups=3)
        ids, w = qf8.route_experts(x, 5, renorm=False)
        dw = torch.randn(tokens, 5, generator=gen, device="cuda")
        got = qf8.route_experts_backward(x, ids, dw, renorm=False).double()
        p = torch.softmax(x.double(), 1)
        full = torch.zeros_like(p).scatter_(1, ids.long(), dw.double())
        want = p * (full - (p * full).sum(1, keepdim=True))
        # fp64 inside, one rounding; fp64 leaves about 2^-50 of the terms
        tol = want.abs() * HALF[dtype] * 1.01 + 2.0 ** -45 * dw.abs().double().max(dim=1, keepdim=True)[0]
        assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("tokens", [2047, 2048, 2049])
@pytest.mark.parametrize("top_k", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine(tokens, top_k, dtype):
    for dim in (8, 2049, 4100):
        x, w, slots, _, _ = combine_case(tokens, 6, top_k, dim, dtype, seed=dim)
        y = qf8.combine_experts(x, w, slots)
        terms = w.double()[:, :, None] * x.double()[slots.long().reshape(-1)].view(tokens, top_k, dim)
        want = terms.sum(1)
        tol = want.abs() * HALF[dtype] * 1.01 + terms.abs().sum(1) * (top_k * 2.0 ** -24)
        assert bool(((y.double() - want).abs() <= tol).all())
