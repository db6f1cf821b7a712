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


@pytest.mark.parametrize("place", [False, True])
def test_norms_at_the_end_of_fp32(place):
    """A finite norm beyond fp32 reads Inf, sets no flag and scales; the largest that fits is itself; Inf among the values is the flag's."""
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    for value, count, fits in ((2.0 ** 127, 1, True), (2.0 ** 127, 3, True), (2.0 ** 127, 4, False), (2.0 ** 120, 1 << 20, False)):
        g = [torch.full((count,), value, device="cuda"), torch.ones(5, device="cuda")]
        out = None if place else [torch.empty_like(t) for t in g]
        norm = value * math.sqrt(count)                       # the ones are below half a step of fp64
        total = qf8.clip_grads(g, 2.0 ** 100, out=out, nonfinite=flag)
        assert total.item() == (float(torch.tensor(norm, dtype=torch.float64).float()) if fits else float("inf")) and flag.item() == 0
        c = torch.tensor(2.0 ** 100 / norm, dtype=torch.float64).float().cuda()
        got = g if place else out
        assert bool((got[0] == value * c).all()) and bool((got[1] == c).all())
        assert qf8.grad_norm([torch.full((count,), value, device="cuda")], nonfinite=flag).isfinite().item() == fits and flag.item() == 0
    g = [torch.tensor([2.0 ** 127, float("inf")], device="cuda")]
    assert qf8.clip_grads(g, 1.0, nonfinite=flag).item() == float("inf") and flag.item() == 1 and g[0][0].item() == 2.0 ** 127
