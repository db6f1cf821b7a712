"""The gated activation and its gradients against the definition in 64 bits.

Tolerances. BF16 inputs: the sigmoid's argument z is rounded a few times, which costs |z| 2^-22 of e^-z, below 2^-15.5
where the result is no subnormal; its slope's two terms, up to |dy b|, are off by 2^-17 of that. FP32 inputs: exp2's argument in two parts,
2^-20 for SiLU; GELU's argument costs |z| 2^-22 there too. Then the type's half step, or a code's (E4M3 2^-4, at least 2^-10; E5M2
2^-3, 2^-17). With FP32 input the codes are quantize_block's of the values bit for bit."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_norm import BF, F32, F8, HALF

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -119          # BF16 inputs: a sigmoid below 2^-126 is 0, where |a| < 88 and so |act| < 88 2^-126 < 2^-119
ACTS = [qf8.ACT_SILU, qf8.ACT_GELU]


def parts(act, a):
    if act == qf8.ACT_SILU:
        s = torch.sigmoid(a)
        return a * s, s + a * s * torch.sigmoid(-a)
    k, m = 2 * math.sqrt(2 / math.pi), 0.044715
    s, t = torch.sigmoid(k * (a + m * a ** 3)), torch.sigmoid(-k * (a + m * a ** 3))
    return a * s, s + a * s * t * k * (1 + 3 * m * a * a)


def made(rows, cols, dtype, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = 2 * torch.randn(rows, 2 * cols, generator=gen, device="cuda")
    x *= 1 + 30 * (torch.rand(1, 2 * cols, generator=gen, device="cuda") < 0.02)
    return x.to(dtype), torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)


def rel(act, dtype):
    return 2.0 ** -20 if act == qf8.ACT_SILU and dtype == F32 else 2.0 ** -15


def near_codes(q, scales, y, slack, fmt):
    """slack: how far the values before the rounding may be off."""
    dt, top, half, least = F8[fmt]
    s = scales.double().repeat_interleave(128, 1)[:, :y.shape[1]]
    v = y * s
    got = q.view(dt).double()
    assert bool(((got - v).abs() <= torch.clamp(half * v.abs(), min=least) * (1 + 2.0 ** -9) + 1.2 * slack * s).all())
    pad = torch.nn.functional.pad(y, (0, -y.shape[1] % 128)).view(y.shape[0], -1, 128).abs().amax(2)
    off = torch.nn.functional.pad(slack, (0, -y.shape[1] % 128)).view(y.shape[0], -1, 128).amax(2)
    want = torch.where(pad > 0, top / pad, 1.0)
    assert bool(((scales - want).abs() <= want * (2.0 ** -22 + 2 * off / pad.clamp(min=TINY))).all())


SIZES = [(1, 8), (1, 128), (3, 136), (64, 256), (17, 1000), (513, 2048), (2, 4104), (4099, 16)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward(rows, cols, act, dtype):
    x, _ = made(rows, cols, dtype, seed=rows + cols)
    fmt = qf8.E5M2 if rows % 3 == 0 else qf8.E4M3
    q, s, y = qf8.gated_act_quantize(x, fmt, act=act, want_y=True)
    a, b = x.double().chunk(2, 1)
    want = parts(act, a)[0] * b
    slack = rel(act, dtype) * want.abs() + TINY * b.abs()
    assert bool(((y.double() - want).abs() <= HALF[dtype] * want.abs() + slack).all())
    near_codes(q, s, want, slack, fmt)
    if dtype == F32:
        q1, s1, _ = qf8.quantize_block(y, 1, 128, fmt, want_amax=False)
        assert torch.equal(q, q1) and torch.equal(s, s1)
    only = qf8.gated_act_quantize(x, fmt, act=act)
    assert only[2] is None and torch.equal(only[0], q) and torch.equal(only[1], s)
    assert torch.equal(qf8.gated_act_quantize(x, None, act=act)[2], y)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward(rows, cols, act, dtype):
    x, dy = made(rows, cols, dtype, seed=rows * 2 + cols)
    codes = cols % 128 == 0
    q, s, dx = qf8.gated_act_backward(dy, x, qf8.E5M2 if codes else None, act=act, want_dx=True)
    a, b = x.double().chunk(2, 1)
    y, slope = parts(act, a)
    d = dy.double()
    want = torch.cat([d * b * slope, d * y], 1)
    slack = torch.cat([rel(act, dtype) * (d * b).abs(), rel(act, dtype) * (d * y).abs() + TINY * d.abs()], 1)
    assert bool(((dx.double() - want).abs() <= HALF[dtype] * want.abs() + slack).all())
    if codes:
        near_codes(q, s, want, slack, qf8.E5M2)
        if dtype == F32:
            q1, s1, _ = qf8.quantize_block(dx, 1, 128, qf8.E5M2, want_amax=False)
            assert torch.equal(q, q1) and torch.equal(s, s1)
        only = qf8.gated_act_backward(dy, x, qf8.E5M2, act=act, pow2_scales=True)
        assert only[2] is None
        if dtype == F32:
            q1, s1, _ = qf8.quantize_block(dx, 1, 128, qf8.E5M2, want_amax=False, pow2_scales=True)
            assert torch.equal(only[0], q1) and torch.equal(only[1], s1)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    """Central differences of the definition in 64 bits, step 2^-20, against FP32 gradients (2^-14 of the terms)."""
    x, dy = made(5, 136, F32, seed=3)
    along = torch.randn(5, 272, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").double()
    dx = qf8.gated_act_backward(dy, x, None, act=act)[2].double()

    def value(t):
        a, b = (x.double() + t * along).chunk(2, 1)
        return float((dy.double() * parts(act, a)[0] * b).sum())
    t = 2.0 ** -20
    slope = (value(t) - value(-t)) / (2 * t)
    assert abs(float((dx * along).sum()) - slope) <= 2.0 ** -14 * float((dx * along).abs().sum())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ends_of_the_range(act, dtype):
    """Far gates, zeros and rows of zeros are finite; Inf and NaN set the flag."""
    a = torch.tensor([0.0, -0.0, 1e4, -1e4, 1e30, -1e30, 100.0, -100.0], device="cuda").repeat(16)
    x = torch.zeros(3, 256, device="cuda")
    x[0, :128], x[0, 128:] = a, 1e-3
    x[2, :128], x[2, 128:] = -200.0, 3.0
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = x.to(dtype)
    q, s, y = qf8.gated_act_quantize(x, qf8.E4M3, act=act, want_y=True, nonfinite=flag)
    dq, ds, dx = qf8.gated_act_backward(torch.ones(3, 128, device="cuda", dtype=dtype), x, qf8.E5M2, act=act, want_dx=True, nonfinite=flag)
    assert flag.item() == 0 and bool(torch.isfinite(y).all()) and bool(torch.isfinite(dx).all())
    assert bool((s[1] == 1).all()) and bool((q[1] == 0).all())
    want = torch.where(a > 1, a, 0.0).to(dtype).double() * x[0, 128].double()
    assert bool(((y[0].double() - want).abs() <= 2 * HALF[dtype] * want.abs() + TINY).all())
    assert bool(((dx[0, :128].double() - torch.where(a.abs() > 1, (a > 1).double(), 0.5) * x[0, 128].double()).abs() <= 2 * HALF[dtype] * 1e-3).all())
    for bad in (float("inf"), float("nan"), float("-inf")):
        z = x.clone()
        z[0, 5] = bad
        flag.zero_()
        qf8.gated_act_quantize(z, qf8.E4M3, act=act, nonfinite=flag)
        assert flag.item() == 1
        flag.zero_()
        dx = qf8.gated_act_backward(torch.ones(3, 128, device="cuda", dtype=dtype), z, None, act=act, want_dx=True, nonfinite=flag)[2]
        if bad != bad:
            assert bool(dx[0, [5, 133]].isnan().all())
        rest = torch.ones(3, 256, dtype=torch.bool, device="cuda")
        rest[0, [5, 133]] = False
        assert flag.item() == 1 and bool(dx[rest].isfinite().all())


def test_sizes_of_nothing_and_refusals():
    e = torch.empty(0, 512, device="cuda", dtype=BF)
    q, s, y = qf8.gated_act_quantize(e, qf8.E4M3, want_y=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and y.shape == (0, 256)
    assert qf8.gated_act_backward(e[:, :256].contiguous(), e, qf8.E4M3)[0].shape == (0, 512)
    x = torch.zeros(4, 272, device="cuda", dtype=BF)
    dy = torch.zeros(4, 136, device="cuda", dtype=BF)
    with pytest.raises(qf8.QF8Error):
        qf8.gated_act_backward(dy, x, qf8.E5M2)             # codes of halves that end inside a group
    with pytest.raises(ValueError):
        qf8.gated_act_quantize(x[:, :271].contiguous(), qf8.E4M3)
    with pytest.raises(ValueError):
        qf8.gated_act_backward(dy[:3], x, None)
    with pytest.raises(TypeError):
        qf8.gated_act_backward(dy.float(), x, None)
    with pytest.raises(ValueError):
        qf8.gated_act_quantize(x, None, q=torch.empty(4, 136, dtype=torch.uint8, device="cuda"))
