"""Scales over the whole range of fp32: the factor 1/Sa * 1/Sb is what counts, not either scale alone.
Bounds as in test_gpu_matmul: the output's rounding, and the sums relative to sum |a||b|."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_matmul import FMT, KIND, assert_close, codes, offsets_of, product, values

pytestmark = pytest.mark.gpu


def far_scales(gen, rows, groups, exponent, pow2):
    """Scales of about 2^exponent in every second row, of about 1 in the others."""
    e = torch.randint(-1, 2, (rows, groups), generator=gen, device="cuda").double()
    e[::2] = e[::2].abs() * (-1.0 if exponent > 0 else 1.0) + exponent
    m = 1.0 if pow2 else 1.0 + 0.99 * torch.rand(rows, groups, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp2(e) * m).float()


@pytest.mark.parametrize("exponent", [-126, -122, -112, -100, 100, 112, 118, 122, 126, 127])
@pytest.mark.parametrize("kind", ["nk", "kn", "groups"])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
def test_scales_of_opposite_magnitude(exponent, kind, fa, fb):
    """One operand's scales near 2^exponent, the other's near 2^-exponent: the results are ordinary numbers."""
    m, n, k = 70, 140, 392
    print(f"range {exponent} {kind} {fa} {fb}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(exponent + 200)
    other = max(-exponent, -126)
    for pow2 in (False, True):
        if exponent == 127 and not pow2:
            continue                                         # 2^127 times a mantissa is still finite, but 1/S is not exact
        a, b = codes(gen, (m, k), fa), codes(gen, (k, n) if kind == "kn" else (n, k), fb)
        g = -(-k // 128)
        if kind == "groups":
            sa, sb = far_scales(gen, m, g, exponent, pow2), far_scales(gen, n, g, other, pow2)
            vb = values(b, sb, fb, 1).t()
        else:
            sa = far_scales(gen, m, g, exponent, pow2)
            sb = far_scales(gen, 2 * b.shape[0], -(-b.shape[1] // 128), other, pow2)[::2][:-(-b.shape[0] // 128)].contiguous()
            vb = values(b, sb, fb, 128)
            vb = vb if kind == "kn" else vb.t()
        ref, mag = product(values(a, sa, fa, 1), vb)
        # half of the rows (and columns) meet scales of about 1: there the factor itself leaves fp32
        ok = (mag < 1e38) & (mag > 1e-30)
        assert bool(ok[::2].any())
        for out_dtype in (torch.float32, torch.bfloat16):
            y = qf8.matmul_block(a, sa, b, sb, FMT[fa], FMT[fb], KIND[kind], pow2_scales=pow2, out_dtype=out_dtype)
            assert_close(y[ok], ref[ok], mag[ok], k, f"{kind} 2^{exponent} pow2={pow2} {out_dtype}")


@pytest.mark.parametrize("exponent", [-120, -104, 104, 120])
def test_weight_gradient_scales_of_opposite_magnitude(exponent):
    counts, m, n = [300, 0, 140], 132, 68
    gen = torch.Generator(device="cuda")
    gen.manual_seed(exponent + 200)
    off = offsets_of(counts, 128)
    g = off[-1] // 128
    for pow2 in (False, True):
        a, sa = codes(gen, (m, off[-1]), "e5m2"), far_scales(gen, m, g, exponent, pow2)
        b, sb = codes(gen, (n, off[-1]), "e4m3"), far_scales(gen, n, g, -exponent, pow2)
        va, vb = values(a, sa, "e5m2", 1), values(b, sb, "e4m3", 1)
        for out_dtype in (torch.float32, torch.bfloat16):
            y = qf8.matmul_block_experts_wgrad(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), qf8.E5M2,
                                               qf8.E4M3, pow2_scales=pow2, out_dtype=out_dtype)
            for e in (0, 2):
                ref, mag = product(va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]].t())
                ok = (mag < 1e38) & (mag > 1e-30)
                assert_close(y[e][ok], ref[ok], mag[ok], off[e + 1] - off[e], f"expert {e} 2^{exponent} pow2={pow2}")
