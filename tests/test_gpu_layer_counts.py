"""The expert layer for a few tokens with every number of tokens to an expert, by the tolerances of its other tests."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_layer_tokens import check, made

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [1, 17, 33, 49])
@pytest.mark.parametrize("dim,hidden", [(272, 144), (128, 256)])
def test_every_number_of_tokens(first, dim, hidden):
    """One expert with all the tokens, and one with all but a few of them, which others share."""
    for tokens in range(first, first + 16):
        alone = torch.ones(tokens, 1, dtype=torch.int32, device="cuda")
        args = made(tokens, dim, hidden, 3, 1, qf8.E4M3, seed=tokens, ids=alone)
        check(qf8.expert_layer_tokens(*args, qf8.E4M3), *args, qf8.E4M3, qf8.ACT_SILU)
        ids = torch.stack([torch.full((tokens,), 2, dtype=torch.int32), torch.arange(tokens, dtype=torch.int32) % 3 - 1], 1).cuda()
        ids[tokens // 2:, 0] = 0 if tokens % 2 else 2
        args = args[:5] + (ids.contiguous(), torch.rand(tokens, 2, device="cuda"))
        check(qf8.expert_layer_tokens(*args, qf8.E4M3, act=qf8.ACT_GELU), *args, qf8.E4M3, qf8.ACT_GELU)
