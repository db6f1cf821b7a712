"""What the expert layer for a few tokens rounds between its inputs and y: nothing that counts beside y's own rounding.

Tolerances. ‖y - exact‖ against ‖rnd_bf16(exact) - exact‖: the activations are rounded to FP16, an eighth of what BF16 is off by, and
the products carry such independent errors to y with their share of its norm: in squares 1 + 1/64, its root 1.008. The sigmoid (2^-17)
and the fp32 sums (about sqrt(n) 2^-25 of the terms' norm) add nothing beside it; 1.02 leaves room for the sample. A BF16 rounding of
the activations has the same size as y's: the root of two."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_gate import ACTS, BF, parts
from test_gpu_layer_tokens import made, values
from test_gpu_norm import F8

pytestmark = pytest.mark.gpu


def exact(x, w1, s1, w2, s2, ids, weights, fmt, act):
    a1, a2 = values(w1, s1, fmt), values(w2, s2, fmt)
    hidden, want = w2.shape[2], torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in range(w1.shape[0]):
        part = (weights.double() * (ids == e)).sum(1, keepdim=True)
        u = x.double() @ a1[e].t()
        want += part * ((parts(act, u[:, :hidden])[0] * u[:, hidden:]) @ a2[e].t())
    return want


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k", [(1, 4096, 512, 16, 8), (4, 1040, 400, 6, 2), (8, 2064, 720, 5, 3), (16, 512, 256, 4, 4),
                                                             (24, 1024, 512, 3, 3), (64, 768, 384, 8, 4), (64, 512, 144, 2, 2)])
@pytest.mark.parametrize("fmt", [qf8.E4M3, qf8.E5M2])
def test_only_y_is_rounded(tokens, dim, hidden, experts, top_k, fmt):
    act = ACTS[tokens % 3 == 1]
    args = made(tokens, dim, hidden, experts, top_k, fmt, seed=tokens * 5 + dim)
    want = exact(*args, fmt, act)
    y = qf8.expert_layer_tokens(*args, fmt, act=act).double()
    rounding = float((want.to(BF).double() - want).norm())
    off = float((y - want).norm())
    assert off <= 1.02 * rounding, f"{off / rounding:.3f} of the rounding of y"


def test_largest_activations():
    """An activation beyond what rounds to a finite BF16 value is held, and its product with a small weight is finite; one that is Inf gives
    Inf, no NaN. Sums of one term, exact: SiLU(93) = 93 in fp32, a = 93 x 2^120, and 93 x 2.75 = 255.75, where BF16 ends at 255."""
    x = torch.zeros(3, 128, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = 93.0, torch.tensor([2.75, 2.0 ** 100, 1.0], device="cuda").to(BF)
    w1 = torch.zeros(1, 256, 128, dtype=torch.uint8, device="cuda")
    w2 = torch.zeros(1, 128, 128, dtype=torch.uint8, device="cuda")
    w1[0, 0, 0], w1[0, 128, 1], w2[0, :, 0] = 0x38, 0x38, 0x38        # the code of 1
    s1, s2 = torch.tensor([1.0, 2.0 ** -120], device="cuda").view(1, 2, 1), torch.full((1, 1, 1), 2.0 ** 10, device="cuda")
    ids, weights = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, 1, device="cuda")
    y = qf8.expert_layer_tokens(x, w1, s1, w2, s2, ids, weights, qf8.E4M3).double()
    assert bool((y[0] == 2.0 ** 118).all()) and bool((y[1] == float("inf")).all()) and bool((y[2] == 93 * 2.0 ** 110).all())


def one_unit(fmt, codes):
    """Weights of one expert by their codes: unit j of both halves takes x[0] and x[1], w2's rows are given."""
    one = 0x38 if fmt == qf8.E4M3 else 0x3C
    dim, hidden = codes.shape
    w1 = torch.zeros(1, 2 * hidden, dim, dtype=torch.uint8, device="cuda")
    w1[0, :hidden, 0], w1[0, hidden:, 1] = one, one
    return w1, torch.ones(1, -(-2 * hidden // 128), -(-dim // 128), device="cuda"), codes[None].contiguous(), torch.ones(1, -(-dim // 128), -(-hidden // 128), device="cuda")


@pytest.mark.parametrize("fmt", [qf8.E4M3, qf8.E5M2])
def test_every_code(fmt):
    """Every code of w2 times one activation, 93: sums of one term, which BF16 rounds once. Inf and NaN codes stay that."""
    codes = torch.zeros(256, 16, dtype=torch.uint8, device="cuda")
    codes[:, 0] = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)
    x = torch.zeros(1, 256, dtype=BF, device="cuda")
    x[0, 0], x[0, 1] = 93.0, 1.0
    ids, weights = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 1, device="cuda")
    y = qf8.expert_layer_tokens(x, *one_unit(fmt, codes), ids, weights, fmt)[0]
    want = (codes[:, 0].contiguous().view(F8[fmt][0]).double() * 93).to(BF)
    assert torch.equal(torch.nan_to_num(y.double(), nan=-1.0, posinf=2e9, neginf=-2e9), torch.nan_to_num(want.double(), nan=-1.0, posinf=2e9, neginf=-2e9))


@pytest.mark.parametrize("fmt", [qf8.E4M3, qf8.E5M2])
@pytest.mark.parametrize("hidden", [16, 80, 128, 272])
def test_activations_of_any_size_side_by_side(fmt, hidden):
    """Activations 93 x 2^p of neighbours, p over all the powers of two that a code has (E4M3 2^-9 to 2^8, E5M2 2^-16 to 2^15), taken out one by
    one: 93 has seven bits, which stay at 2^-31 of the largest neighbour. Before and behind, experts that the token did not choose."""
    top, low = (8, 9) if fmt == qf8.E4M3 else (15, 16)
    p = torch.randint(-low, top + 1, (hidden,), generator=torch.Generator().manual_seed(hidden))
    power = torch.tensor([2.0 ** int(i) for i in p], dtype=torch.float64).cuda()
    eye = torch.zeros(hidden, hidden, dtype=torch.uint8, device="cuda")
    eye[range(hidden), range(hidden)] = 0x38 if fmt == qf8.E4M3 else 0x3C
    w1, s1, w2, s2 = (t.repeat(3, *[1] * (t.dim() - 1)) for t in one_unit(fmt, eye))
    w1[1, hidden:, 1] = power.float().to(F8[fmt][0]).view(torch.uint8)
    x = torch.zeros(5, hidden, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = 93.0, torch.tensor([1.0, 2.0 ** 60, 2.0 ** -60, 0.0, 2.0 ** 97]).to(BF).cuda()
    ids, weights = torch.ones(5, 1, dtype=torch.int32, device="cuda"), torch.ones(5, 1, device="cuda")
    y = qf8.expert_layer_tokens(x, w1, s1, w2, s2, ids, weights, fmt).double()
    assert torch.equal(y, 93 * power[None] * x[:, 1:2].double())


@pytest.mark.parametrize("fmt", [qf8.E4M3, qf8.E5M2])
def test_activations_and_scales_of_any_size(fmt):
    """93 x 2^p under scales 2^s, from small by large to large by small: exact. One call for each s, one token for each p."""
    eye = torch.zeros(32, 32, dtype=torch.uint8, device="cuda")
    eye[range(32), range(32)] = 0x38 if fmt == qf8.E4M3 else 0x3C
    w1, s1, w2, _ = one_unit(fmt, eye)
    for s in (-100, -70, -30, 0, 30, 70, 100, 120):
        powers = [p for p in range(-118, 119, 4) if -118 <= p - s <= 118]
        x = torch.zeros(len(powers), 32, dtype=BF, device="cuda")
        x[:, 0], x[:, 1] = 93.0, torch.tensor([2.0 ** p for p in powers], dtype=torch.float64).to(BF).cuda()
        ids, weights = torch.zeros(len(powers), 1, dtype=torch.int32, device="cuda"), torch.ones(len(powers), 1, device="cuda")
        y = qf8.expert_layer_tokens(x, w1, s1, w2, torch.full((1, 1, 1), 2.0 ** s, device="cuda"), ids, weights, fmt).double()
        want = torch.tensor([93 * 2.0 ** (p - s) for p in powers], dtype=torch.float64).cuda()[:, None].expand(-1, 32)
        assert torch.equal(y, want), s
