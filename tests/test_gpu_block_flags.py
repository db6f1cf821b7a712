"""The flag of results that are not finite where only their rounding to BF16 is: 255.5 x 2^120 is the first value that BF16 rounds to Inf.
Codes alone saturate, and FP32 results hold the value."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def flagged(call):
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(flag)
    return flag.item(), out


@pytest.mark.parametrize("b,inf", [(2.75, True), (2.734375, False)])          # 93 times these: 255.75 and 254.3
def test_gate(b, inf):
    x = torch.zeros(2, 256, device="cuda")
    x[1, 5], x[1, 133] = 93.0, b * 2.0 ** 120
    set_, (_, _, y) = flagged(lambda f: qf8.gated_act_quantize(x.to(BF), qf8.E4M3, want_y=True, nonfinite=f))
    assert set_ == inf and bool(y.isinf().any()) == inf
    assert flagged(lambda f: qf8.gated_act_quantize(x.to(BF), qf8.E4M3, nonfinite=f))[0] == 0
    set_, (_, _, y) = flagged(lambda f: qf8.gated_act_quantize(x, qf8.E4M3, want_y=True, nonfinite=f))
    assert set_ == 0 and bool(y.isfinite().all())
    one = torch.zeros(2, 256, device="cuda", dtype=BF)                       # gradients: dy act(a), dy b act'(a)
    one[1, 5], one[1, 133] = 93.0, 1.0
    dy = torch.zeros(2, 128, device="cuda", dtype=BF)
    dy[1, 5] = b * 2.0 ** 120
    set_, (_, _, dx) = flagged(lambda f: qf8.gated_act_backward(dy, one, qf8.E5M2, want_dx=True, nonfinite=f))
    assert set_ == inf and bool(dx.isinf().any()) == inf
    assert flagged(lambda f: qf8.gated_act_backward(dy, one, qf8.E5M2, nonfinite=f))[0] == 0


@pytest.mark.parametrize("weight,inf", [(150.0, True), (149.0, False)])       # 2 / sqrt(11 / 8) times these: 255.8 and 254.1
def test_norm(weight, inf):
    x = torch.ones(3, 8, device="cuda")
    x[2, 0] = 2.0
    w = torch.ones(8, device="cuda")
    w[0] = weight * 2.0 ** 120
    set_, got = flagged(lambda f: qf8.rms_norm_quantize(x.to(BF), w, qf8.E4M3, want_y=True, nonfinite=f))
    assert set_ == inf and bool(got.y.isinf().any()) == inf
    assert flagged(lambda f: qf8.rms_norm_quantize(x.to(BF), w, qf8.E4M3, nonfinite=f))[0] == 0
    set_, got = flagged(lambda f: qf8.rms_norm_quantize(x, w, qf8.E4M3, want_y=True, nonfinite=f))
    assert set_ == 0 and bool(got.y.isfinite().all())
