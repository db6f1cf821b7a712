"""The norm over many tensors and their scaling. Sums are fp64, so the norm is the exact one rounded to fp32 (half a step 2^-24, and
2^-40 for the sums); an output is its gradient times the fp32 factor, rounded once, bit for bit for the factor or a neighbour of it (the
factor's own rounding may fall to the other side)."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def made(sizes, types, seed=0, scale=1e-2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [(scale * (1 + i % 5) * torch.randn(n, generator=gen, device="cuda")).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def exact(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check_outputs(out, grads, norm, max_norm):
    c = torch.tensor(min(1.0, max_norm / (norm + 1e-6)), dtype=torch.float64).float()
    near = [c] if c == 1 else [c, torch.nextafter(c, torch.zeros(())), torch.nextafter(c, torch.ones(()))]
    assert any(all(torch.equal(o, (g.float() * f.cuda()).to(g.dtype)) for o, g in zip(out, grads)) for f in near)


@pytest.mark.parametrize("sizes", [[1], [7], [0, 5, 0], [16384], [16385], [100000, 3, 17], [5, 8, 16, 64, 100] * 60, [2000003, 1]])
@pytest.mark.parametrize("types", [[BF], [F32], [BF, F32, F32]])
@pytest.mark.parametrize("fraction", [0.3, 2.0])
def test_clip(sizes, types, fraction):
    grads = made(sizes, types, seed=len(sizes))
    norm = exact(grads)
    keep = [g.clone() for g in grads]
    out = [torch.full_like(g, 7) for g in grads]
    got = qf8.clip_grads(grads, fraction * norm, out=out)
    assert abs(got.item() - norm) <= (2.0 ** -24 + 2.0 ** -40) * norm
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    check_outputs(out, grads, norm, fraction * norm)
    assert torch.equal(qf8.grad_norm(grads), got)
    place = [g.clone() for g in grads]
    assert torch.equal(qf8.clip_grads(place, fraction * norm), got)
    assert all(torch.equal(a, b) for a, b in zip(place, out))


def test_any_alignment_and_shape():
    """Views at odd addresses beside others, and tensors of any number of dimensions; what lies between stays."""
    base = torch.randn(300000, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(BF)
    flat = torch.randn(100000, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    cuts = [(1, 50000), (50001, 33333), (83340, 17), (90000, 131072)]
    grads = [base[a:a + n] for a, n in cuts] + [flat[1:60001].view(300, 200), flat[60003:60004], flat[60010:].view(-1, 10)[None]]
    norm = exact(grads)
    before, fbefore = base.clone(), flat.clone()
    want = [g.clone() for g in grads]
    qf8.clip_grads(grads, 0.5 * norm)
    check_outputs(grads, want, norm, 0.5 * norm)
    mask = torch.ones_like(base, dtype=torch.bool)
    for a, n in cuts:
        mask[a:a + n] = False
    assert torch.equal(base[mask], before[mask]) and flat[0] == fbefore[0] and torch.equal(flat[60001:60003], fbefore[60001:60003])


def test_range():
    """Squares beyond fp32 and below it; a norm beyond fp32; no values at all."""
    big = [torch.full((1000,), 1e30, device="cuda"), torch.full((10,), 3e38, device="cuda")]
    norm = exact(big)
    out = [torch.empty_like(g) for g in big]
    assert qf8.clip_grads(big, 1.0, out=out).item() == float("inf") or abs(qf8.grad_norm(big).item() - norm) <= 2.0 ** -23 * norm
    check_outputs(out, big, norm, 1.0)
    tiny = [torch.full((1000,), 1e-38, device="cuda")]
    assert abs(qf8.grad_norm(tiny).item() - exact(tiny)) <= 2.0 ** -23 * exact(tiny)
    zero = [torch.zeros(100, device="cuda"), torch.empty(0, device="cuda")]
    assert qf8.clip_grads(zero, 1.0).item() == 0 and bool((zero[0] == 0).all())
    assert qf8.grad_norm([torch.empty(0, device="cuda")]).item() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_not_finite(bad, dtype):
    grads = made([20000, 33], [dtype])
    grads[1][7] = bad
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(g) for g in grads]
    norm = qf8.clip_grads(grads, 1e-3, out=out, nonfinite=flag)
    assert not math.isfinite(norm.item()) and flag.item() == 1
    bits = torch.int16 if dtype == BF else torch.int32
    assert all(torch.equal(o.view(bits), g.view(bits)) for o, g in zip(out, grads))
    flag.zero_()
    grads[1][7] = 0
    qf8.clip_grads(grads, 1e-3, nonfinite=flag)
    assert flag.item() == 0


def test_many_tensors_and_sums_of_many_chunks():
    grads = made([3 + i % 50 for i in range(1000)] + [30_000_001], [F32, BF], seed=5)
    norm = exact(grads)
    got = qf8.clip_grads(grads, 0.1 * norm, out=[torch.empty_like(g) for g in grads])
    assert abs(got.item() - norm) <= (2.0 ** -24 + 2.0 ** -40) * norm


def test_refusals():
    g = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError):
        qf8.clip_grads([g.t()[:, :4]], 1.0)
    with pytest.raises(TypeError):
        qf8.clip_grads([g.half()], 1.0)
    with pytest.raises(ValueError):
        qf8.clip_grads([g], 1.0, out=[torch.zeros(64, device="cuda")])
    with pytest.raises(TypeError):
        qf8.clip_grads([g], 1.0, out=[torch.zeros(8, 8, device="cuda", dtype=BF)])
    with pytest.raises(TypeError):
        qf8.clip_grads([g, torch.zeros(3)], 1.0)
    with pytest.raises(ValueError):
        qf8.clip_grads([g, g], 1.0)
    e = torch.empty(0, device="cuda")
    assert qf8.clip_grads([e, e], 1.0).item() == 0 and qf8.grad_norm([g, g]).item() == 0
    with pytest.raises(qf8.QF8Error):
        qf8.clip_grads([g], 0.0)
    with pytest.raises(qf8.QF8Error):
        qf8.clip_grads([g], 1.0, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
