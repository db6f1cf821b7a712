"""BF16 results of fp32 sums. Bounds as those of FP32 results in test_gpu_matmul: half a step of the result, and
per group at most 128 additions, taken as a whole step (2^-23) each, one fp32 addition and three roundings of the
factor, relative to sum |a||b|."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_matmul import DT, FMT, KIND, codes, guarded, offsets_of, operands, product, scales, values

pytestmark = pytest.mark.gpu


def assert_fp32_sums(y, ref, mag, k, what):
    tol = ref.abs() * 2.0 ** -8 * 1.01 + mag * ((2 * 128 + -(-k // 128) + 8) * 2.0 ** -24) + 1e-40
    bad = ~((y.double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


@pytest.mark.parametrize("m,n,k", [(1, 4, 4), (17, 20, 132), (100, 301, 516), (129, 260, 400), (333, 517, 388), (8, 2052, 8200),
                                   (2000, 2100, 640)])
@pytest.mark.parametrize("kind", ["nk", "kn", "groups"])
@pytest.mark.parametrize("pow2", [False, True])
def test_sizes(m, n, k, kind, pow2):
    n = n // 4 * 4 if kind == "kn" else n
    print(f"fp32 sums {kind} {m}x{n}x{k} pow2={pow2}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m + n + k)
    a, sa = codes(gen, (m, k), "e4m3"), scales(gen, (m, -(-k // 128)), pow2)
    b, sb, vb = operands(gen, kind, n, k, "e5m2", pow2)
    y, after = guarded((m, n), torch.bfloat16)
    qf8.matmul_block(a, sa, b, sb, qf8.E4M3, qf8.E5M2, KIND[kind], pow2_scales=pow2, out=y, fp32_sums=True)
    torch.cuda.synchronize()
    assert bool((after == 77.0).all()), "written past the output"
    ref, mag = product(values(a, sa, "e4m3", 1), vb)
    assert_fp32_sums(y, ref, mag, k, kind)
    full = qf8.matmul_block(a, sa, b, sb, qf8.E4M3, qf8.E5M2, KIND[kind], pow2_scales=pow2, out_dtype=torch.float32)
    assert torch.equal(y, full.to(torch.bfloat16))           # the same sums, rounded once


@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3")])
@pytest.mark.parametrize("kind", ["nk", "kn", "groups"])
def test_sums_that_cancel(fa, fb, kind):
    """Beside two large products that cancel every small one counts: all sums are whole numbers below 2^24."""
    m, n, k = 36, 72, 512
    a = torch.full((m, k), 1.0, device="cuda")
    a[:, ::8] = a[:, 1::8] = 448.0
    b = torch.full((n, k), 1.0, device="cuda")
    b[:, ::8], b[:, 1::8] = 448.0, -448.0
    b[::3, 5::8] = 3.0
    a[::2, 6::8] = -5.0
    want = (a.double() @ b.double().t()).to(torch.bfloat16)
    qa, qb = a.to(DT[fa]).view(torch.uint8), b.to(DT[fb]).view(torch.uint8)
    assert torch.equal(qa.view(DT[fa]).float(), a) and torch.equal(qb.view(DT[fb]).float(), b)
    one = lambda *s: torch.ones(*s, device="cuda")
    sb = one(n, 4) if kind == "groups" else one(1, 4) if kind == "nk" else one(4, 1)
    qb = qb.t().contiguous() if kind == "kn" else qb
    for pow2 in (False, True):
        y = qf8.matmul_block(qa, one(m, 4), qb, sb, FMT[fa], FMT[fb], KIND[kind], pow2_scales=pow2, fp32_sums=True)
        assert torch.equal(y, want)


@pytest.mark.parametrize("kind", ["nk", "kn"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("pow2", [False, True])
def test_experts(kind, gather, pow2):
    counts, n, k = [5, 0, 17, 1, 64, 130], 148, 272
    print(f"fp32 sums experts {kind} gather={gather} pow2={pow2}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    off = [3 + o for o in offsets_of(counts)]
    nrows, tokens = off[-1] + 9, 40 if gather else off[-1] + 9
    a, sa = codes(gen, (tokens, k), "e4m3"), scales(gen, (tokens, 3), pow2)
    each = [operands(gen, kind, n, k, "e4m3", pow2) for _ in counts]
    rows = torch.randint(-1, tokens, (nrows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    y, after = guarded((nrows, n), torch.bfloat16)
    qf8.matmul_block_experts(a, sa, torch.stack([e[0] for e in each]), torch.stack([e[1] for e in each]),
                             torch.tensor(off, dtype=torch.int32, device="cuda"), qf8.E4M3, qf8.E4M3, KIND[kind], rows=rows,
                             pow2_scales=pow2, out=y, fp32_sums=True)
    torch.cuda.synchronize()
    assert bool((after == 77.0).all()) and bool((y[:3] == 0).all()) and bool((y[off[-1]:] == 0).all())
    va = values(a, sa, "e4m3", 1)
    if gather:
        va = torch.where((rows >= 0)[:, None], va[rows.clamp_min(0).long()], 0.0)
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, mag = product(va[lo:hi], each[e][2])
            assert_fp32_sums(y[lo:hi], ref, mag, k, f"expert {e}")


@pytest.mark.parametrize("m,n", [(68, 132), (257, 21)])
@pytest.mark.parametrize("pow2", [False, True])
def test_weight_gradient(m, n, pow2):
    counts = [128, 0, 256, 5]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m)
    off = offsets_of(counts, 128)
    a, sa = codes(gen, (m, off[-1]), "e5m2"), scales(gen, (m, off[-1] // 128), pow2)
    b, sb = codes(gen, (n, off[-1]), "e4m3"), scales(gen, (n, off[-1] // 128), pow2)
    y, after = guarded((len(counts), m, n), torch.bfloat16)
    qf8.matmul_block_experts_wgrad(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), qf8.E5M2, qf8.E4M3,
                                   pow2_scales=pow2, out_dtype=torch.bfloat16, out=y, fp32_sums=True)
    torch.cuda.synchronize()
    assert bool((after == 77.0).all())
    va, vb = values(a, sa, "e5m2", 1), values(b, sb, "e4m3", 1)
    for e in range(len(counts)):
        ref, mag = product(va[:, off[e]:off[e + 1]], vb[:, off[e]:off[e + 1]].t())
        assert_fp32_sums(y[e], ref, mag, max(1, off[e + 1] - off[e]), f"expert {e}")
