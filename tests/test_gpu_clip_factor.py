"""The factor of clipping, bit for bit: whole numbers, whose squares' sum is exact, so N is the fp64 root and the factor its quotient, rounded
to fp32 once, whatever the largest norm is."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [1.0, 0.1, 1 / 3, 7.3, math.pi * 100, 12345.678, 2e-46])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_factor(max_norm, dtype):
    gen = torch.Generator(device="cuda").manual_seed(7)
    grads = [torch.randint(-255, 256, (n,), generator=gen, device="cuda").to(dtype) for n in (100003, 17, 4096)]
    norm = math.sqrt(sum(int(g.long().square().sum()) for g in grads))
    c = torch.tensor(min(1.0, max_norm / (norm + 1e-6)), dtype=torch.float64).float().cuda()
    out = [torch.empty_like(g) for g in grads]
    got = qf8.clip_grads(grads, max_norm, out=out)
    assert got.item() == float(torch.tensor(norm, dtype=torch.float64).float())
    for g, o in zip(grads, out):
        assert torch.equal(o, (g.float() * c).to(dtype))
