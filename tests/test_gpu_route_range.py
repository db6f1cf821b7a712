"""The choice of experts at the ends of the range."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_experts import SCORE

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
