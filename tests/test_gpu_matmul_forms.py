"""Forms of the experts' products that the other files leave out: FP32 results with gathered rows in both layouts,
BF16 weight gradients. Bounds as in test_gpu_matmul."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_matmul import assert_close, codes, guarded, offsets_of, product, scales, values
from test_gpu_matmul_rows import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[1] * 40, [33, 0, 257, 2]])
@pytest.mark.parametrize("kind", ["nk", "kn"])
@pytest.mark.parametrize("k", [100, 256, 1000])
def test_fp32_results_of_experts(counts, kind, k):
    """FP32 results of gathered rows, some of no source, with a ragged sum and power-of-two scales."""
    for pow2 in (False, True):
        for gather in (False, True):
            run(0, counts, 5, kind, torch.float32, gather, pow2, n=260, k=k)


@pytest.mark.parametrize("counts", [[128, 0, 256, 5], [300, 7, 140]])
@pytest.mark.parametrize("m,n", [(68, 132), (257, 21), (640, 520)])
@pytest.mark.parametrize("pow2", [False, True])
def test_weight_gradient_in_bf16(counts, m, n, pow2):
    """BF16 weight gradients of experts: planes of rows that do not start at an even element."""
    print(f"experts wgrad bf16 {counts} {m}x{n} pow2={pow2}", flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(m + n)
    off = offsets_of(counts, 128)
    nrows = off[-1] + 128
    a, sa = codes(gen, (m, nrows), "e5m2"), scales(gen, (m, nrows // 128), pow2)
    b, sb = codes(gen, (n, nrows), "e4m3"), scales(gen, (n, nrows // 128), pow2)
    y, after = guarded((len(counts), m, n), torch.bfloat16)
    qf8.matmul_block_experts_wgrad(a, sa, b, sb, torch.tensor(off, dtype=torch.int32, device="cuda"), qf8.E5M2, qf8.E4M3,
                                   pow2_scales=pow2, out_dtype=torch.bfloat16, out=y)
    torch.cuda.synchronize()
    assert bool((after == 77.0).all()), "written past the output"
    va, vb = values(a, sa, "e5m2", 1), values(b, sb, "e4m3", 1)
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, mag = product(va[:, lo:hi], vb[:, lo:hi].t())
            assert_close(y[e], ref, mag, hi - lo, f"expert {e}")
        else:
            assert bool((y[e] == 0).all())
