"""R = 1 / sqrt(mean + eps) of the norm, where the sum of squares is exact in fp32: the mean with eps rounded once or twice (2^-24 each, half
of it in R) and the root to half a step, 2^-24: 2^-23 of R, and 1.5 2^-24 where eps is below 2^-24 of the mean."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [8, 136, 1000, 1032, 2056, 4104, 5128, 7168, 10008])
@pytest.mark.parametrize("rows", [700, 5])
def test_root(rows, cols):
    """Whole numbers up to 31: squares and their sums are below 2^24 in any order."""
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randint(-31, 32, (rows, cols), generator=gen, device="cuda").to(torch.bfloat16)
    x[:, 0] = torch.randint(1, 32, (rows,), generator=gen, device="cuda").to(torch.bfloat16)
    w = torch.ones(cols, device="cuda")
    for eps, tol in ((2.0 ** -40, 1.5 * 2.0 ** -24), (1e-6, 2.0 ** -23), (3.0, 2.0 ** -23)):
        got = qf8.rms_norm_quantize(x, w, qf8.E4M3, eps=eps, want_rstd=True).rstd.double()
        eps = float(torch.tensor(eps, dtype=torch.float32))
        want = (x.double().square().sum(1) / cols + eps).rsqrt()
        assert float(((got - want).abs() / want).max()) <= tol * (1 + 2.0 ** -18)


@pytest.mark.parametrize("cols,value", [(8, 6.3e18), (264, 1.1e18), (264, 1e19), (16384, 1.0)])
def test_mean_and_eps_beyond_fp32(cols, value):
    """The largest eps: the mean with it overflows fp32 where the sum of squares does not, or does, or is nothing beside it. R is rounded
    once from fp64, or half an ulp from its fp32 argument: 2^-23; y has two more roundings, and its subnormals half a step 2^-150."""
    eps = torch.finfo(torch.float32).max
    x = torch.full((3, cols), value, device="cuda")
    x[1] *= -0.5
    got = qf8.rms_norm_quantize(x, torch.ones(cols, device="cuda"), None, eps=eps, want_rstd=True)
    want = (x.double().square().mean(1) + eps).rsqrt()
    assert bool(((got.rstd.double() - want).abs() <= 2.0 ** -23 * (1 + 2.0 ** -18) * want).all())
    y = x.double() * want[:, None]
    assert bool(((got.y.double() - y).abs() <= 2.0 ** -22 * y.abs() + 2.0 ** -150).all())
