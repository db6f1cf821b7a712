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
