"""Tensors of more than 2^32 bytes and values: their last rows against the same rows on their own, and the largest weights of the
expert layer for a few tokens."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_gate import BF, parts
from test_gpu_layer_tokens import blocks
from test_gpu_norm import F8

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def tail(rows, cols, last, seed):
    """Zeros but for the last rows."""
    t = torch.zeros(rows, cols, device="cuda", dtype=BF)
    t[-last:] = torch.randn(last, cols, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)
    return t


def test_norm():
    rows, cols = (1 << 18) + 5, 16384                       # 2^32 values and some
    x, w = tail(rows, cols, 6, 1), torch.ones(cols, device="cuda")
    got = qf8.rms_norm_quantize(x, w, qf8.E4M3, want_rstd=True)
    want = qf8.rms_norm_quantize(x[-6:].contiguous(), w, qf8.E4M3, want_rstd=True)
    for g, v in ((got.q, want.q), (got.scales, want.scales), (got.rstd, want.rstd)):
        assert torch.equal(g[-6:], v)
    assert bool((got.q[-7] == 0).all()) and bool((got.scales[-7] == 1).all())
    rstd = got.rstd
    del got
    dx, dw = qf8.rms_norm_backward(x, x, rstd, w)
    ox, ow = qf8.rms_norm_backward(x[-6:].contiguous(), x[-6:].contiguous(), rstd[-6:].contiguous(), w)
    assert torch.equal(dx[-6:], ox) and bool((dx[-7] == 0).all())
    assert bool(((dw - ow).abs() <= 2.0 ** -20 * ow.abs() + 1e-5).all())


def test_gate():
    rows, cols = (1 << 20) + 3, 2048                        # 2^32 values and some
    x, dy = tail(rows, 2 * cols, 5, 2), tail(rows, cols, 5, 3)
    q, s, _ = qf8.gated_act_quantize(x, qf8.E4M3)
    wq, ws, _ = qf8.gated_act_quantize(x[-5:].contiguous(), qf8.E4M3)
    assert torch.equal(q[-5:], wq) and torch.equal(s[-5:], ws) and bool((q[-6] == 0).all())
    del q, s
    q, s, _ = qf8.gated_act_backward(dy, x, qf8.E5M2)
    wq, ws, _ = qf8.gated_act_backward(dy[-5:].contiguous(), x[-5:].contiguous(), qf8.E5M2)
    assert torch.equal(q[-5:], wq) and torch.equal(s[-5:], ws)


def test_clip():
    n = (1 << 32) + 13
    g = torch.zeros(n, device="cuda", dtype=BF)
    g[-20:] = 2.0
    g[0] = 4.0
    norm = (20 * 4 + 16) ** 0.5
    assert abs(qf8.clip_grads([g], 0.5 * norm).item() - norm) <= 2.0 ** -23 * norm
    assert bool((g[-20:] == 1).all()) and g[0] == 2 and bool((g[1:1000] == 0).all()) and bool((g[-1000:-20] == 0).all())


def test_experts_beyond_four_gigabytes():
    gen = torch.Generator(device="cuda").manual_seed(4)
    one1, sc1 = blocks(gen, 1, 8192, 8192, qf8.E4M3)
    one2, sc2 = blocks(gen, 1, 8192, 4096, qf8.E4M3)
    w1 = torch.zeros(70, 8192, 8192, dtype=torch.uint8, device="cuda")
    w2 = torch.zeros(140, 8192, 4096, dtype=torch.uint8, device="cuda")[:70]
    s1, s2 = torch.ones(70, 64, 64, device="cuda"), torch.ones(70, 64, 32, device="cuda")
    w1[69], s1[69], w2[69], s2[69] = one1[0], sc1[0], one2[0], sc2[0]
    x = torch.randn(3, 8192, generator=gen, device="cuda").to(BF)
    weights = torch.rand(3, 2, generator=gen, device="cuda")
    ids = torch.tensor([[69, 0], [3, 69], [1, 2]], dtype=torch.int32, device="cuda")
    y = qf8.expert_layer_tokens(x, w1, s1, w2, s2, ids, weights, qf8.E4M3)
    only = torch.tensor([[0, -1], [-1, 0], [-1, -1]], dtype=torch.int32, device="cuda")
    want = qf8.expert_layer_tokens(x, one1, sc1, one2, sc2, only, weights, qf8.E4M3)
    # the same products, cut at other places of the run: fp32 sums of 4096 terms, and a step of the rounding to BF16
    assert float((y.float() - want.float()).norm()) <= 2.0 ** -8 * float(want.float().norm()) and bool((y[2] == 0).all())


def test_largest_weights():
    """dim and hidden at their largest: a weight of 2^31 codes. Element by element as in the tests of smaller layers: BF16's half
    steps of the activations and of y, and the fp32 sums."""
    n = 32768
    gen = torch.Generator(device="cuda").manual_seed(5)
    q1 = torch.randint(0, 256, (1, 2 * n, n), dtype=torch.uint8, generator=gen, device="cuda")
    q1 = torch.where((q1 & 0x7F) < 0x70, q1, 0)             # values up to 120
    q2 = torch.randint(0, 256, (1, n, n), dtype=torch.uint8, generator=gen, device="cuda")
    q2 = torch.where((q2 & 0x7F) < 0x70, q2, 0)
    s1 = 4000.0 + 1000 * torch.rand(1, 2 * n // 128, n // 128, generator=gen, device="cuda")
    s2 = 4000.0 + 1000 * torch.rand(1, n // 128, n // 128, generator=gen, device="cuda")
    x = torch.randn(1, n, generator=gen, device="cuda").to(BF)
    ids, weights = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    y = qf8.expert_layer_tokens(x, q1, s1, q2, s2, ids, weights, qf8.E4M3)[0].double()

    def product(q, s, v, i):
        w = q[0, i:i + 2048].view(F8[qf8.E4M3][0]).double()
        w /= s[0, i // 128:i // 128 + 16].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w @ v, w.abs() @ v.abs()
    both = [product(q1, s1, x[0].double(), i) for i in range(0, 2 * n, 2048)]
    u, size = torch.cat([b[0] for b in both]), n * 2.0 ** -24 * torch.cat([b[1] for b in both])
    f = parts(qf8.ACT_SILU, u[:n])[0]
    a = f * u[n:]
    da = 1.13 * size[:n] * u[n:].abs() + f.abs() * size[n:] + (2.0 ** -15 + 2.0 ** -8 + n * 2.0 ** -24) * a.abs()
    for i in range(0, n, 2048):
        want, _ = product(q2, s2, a, i)
        off = product(q2, s2, da, i)[1]
        assert bool(((y[i:i + 2048] - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * off).all())
