"""Rows that belong to no expert, before the first one as well as after the last. Bounds as in
test_gpu_matmul: the output's rounding, and the sums relative to sum |a||b|."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_matmul import KIND, assert_close, codes, guarded, offsets_of, operands, product, scales, values

pytestmark = pytest.mark.gpu


def run(first, counts, tail, kind, out_dtype, gather=False, pow2=False, n=148, k=272):
    experts = len(counts)
    print(f"experts from row {first} {counts[:8]} {kind} {out_dtype} gather={gather} pow2={pow2}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(first + experts)
    off = [first + o for o in offsets_of(counts)]
    nrows = off[-1] + tail
    tokens = 40 if gather else nrows
    a, sa = codes(gen, (tokens, k), "e4m3"), scales(gen, (tokens, -(-k // 128)), pow2)
    each = [operands(gen, kind, n, k, "e4m3", pow2) for _ in range(min(experts, 6))]
    at = [each[e % len(each)] for e in range(experts)]
    rows = torch.randint(-2, tokens + 2, (nrows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    y, after = guarded((nrows, n), out_dtype)
    qf8.matmul_block_experts(a, sa, torch.stack([e[0] for e in at]), torch.stack([e[1] for e in at]),
                             torch.tensor(off, dtype=torch.int32, device="cuda"), qf8.E4M3, qf8.E4M3, KIND[kind], rows=rows,
                             pow2_scales=pow2, out_dtype=out_dtype, out=y)
    torch.cuda.synchronize()
    assert bool((after == 77.0).all()), "written past the output"
    assert bool((y[:first] == 0).all()), "rows before the first expert"
    assert bool((y[off[-1]:] == 0).all()), "rows after the last expert"
    va = values(a, sa, "e4m3", 1)
    if gather:
        ok = (rows >= 0) & (rows < tokens)
        va = torch.where(ok[:, None], va[rows.clamp(0, tokens - 1).long()], 0.0)
    for e in range(experts):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, mag = product(va[lo:hi], at[e][2])
            assert_close(y[lo:hi], ref, mag, k, f"expert {e}")


@pytest.mark.parametrize("first", [1, 40, 300])
@pytest.mark.parametrize("kind", ["nk", "kn"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gather", [False, True])
def test_rows_before_the_first_expert(first, kind, out_dtype, gather):
    for pow2 in (False, True):
        run(first, [5, 0, 17, 130], 9, kind, out_dtype, gather, pow2)
    run(first, [0, 0], 0, kind, out_dtype, gather)


@pytest.mark.parametrize("experts", [1, 62, 63, 64, 65, 129])
def test_many_experts_after_other_rows(experts):
    run(70, [1 + e % 5 for e in range(experts)], 3, "nk", torch.bfloat16, n=36, k=132)


@pytest.mark.parametrize("kind", ["nk", "kn"])
def test_large_tiles_after_other_rows(kind):
    run(259, [700, 0, 1100, 513, 900, 623], 300, kind, torch.bfloat16, n=2052, k=384)
    run(259, [700, 0, 1100, 513, 900, 623], 300, kind, torch.float32, n=2052, k=384)


def test_a_share_of_the_experts():
    """A slice of the weights with the same slice of the offsets: the other experts' rows are zeros."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    off = torch.tensor(offsets_of([30, 40, 0, 50, 60]), dtype=torch.int32, device="cuda")
    a, sa = codes(gen, (180, 256), "e4m3"), scales(gen, (180, 2), False)
    each = [operands(gen, "nk", 132, 256, "e4m3", False) for _ in range(5)]
    b, sb = torch.stack([e[0] for e in each]), torch.stack([e[1] for e in each])
    whole = qf8.matmul_block_experts(a, sa, b, sb, off, qf8.E4M3, qf8.E4M3)
    total = torch.zeros_like(whole)
    for lo, hi in ((0, 2), (2, 4), (4, 5)):
        part = torch.full_like(whole, float("nan"))
        qf8.matmul_block_experts(a, sa, b[lo:hi], sb[lo:hi], off[lo:hi + 1], qf8.E4M3, qf8.E4M3, out=part)
        total += part
    assert torch.equal(total, whole)
