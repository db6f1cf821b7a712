"""The whole expert layer for a few tokens against its definition in 64 bits.

Tolerances, element by element: a product's fp32 sum of n terms is off by n 2^-24 of the sum of their magnitudes; the
activation by 2^-15 of itself (its slope is at most 1.13) and, rounded to BF16, by its half step 2^-8; y by the sums of all
that under |W2| and the weights, and its own half step."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_gate import ACTS, BF, parts
from test_gpu_norm import F8

pytestmark = pytest.mark.gpu


def blocks(gen, experts, n, k, fmt):
    w = torch.randn(experts, n, k, generator=gen, device="cuda") * k ** -0.5
    w *= torch.exp(torch.randn(experts, 1, k, generator=gen, device="cuda") * 0.3)
    made = [qf8.quantize_block(e, 128, 128, fmt, want_amax=False)[:2] if k % 4 == 0 else None for e in w]
    return torch.stack([q for q, _ in made]), torch.stack([s for _, s in made])


def values(q, s, fmt):
    v = q.view(F8[fmt][0]).double()
    return v / s.double().repeat_interleave(128, 1)[:, :v.shape[1]].repeat_interleave(128, 2)[:, :, :v.shape[2]]


def made(tokens, dim, hidden, experts, top_k, fmt, seed=0, ids=None):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(tokens, dim, generator=gen, device="cuda").to(BF)
    w1, s1 = blocks(gen, experts, 2 * hidden, dim, fmt)
    w2, s2 = blocks(gen, experts, dim, hidden, fmt)
    if ids is None:
        ids = torch.rand(tokens, experts, generator=gen, device="cuda").argsort(1)[:, :top_k].to(torch.int32).contiguous()
    weights = torch.rand(ids.shape, generator=gen, device="cuda")
    return x, w1, s1, w2, s2, ids, weights


def check(y, x, w1, s1, w2, s2, ids, weights, fmt, act):
    hidden, dim = w2.shape[2], w2.shape[1]
    a1, a2 = values(w1, s1, fmt), values(w2, s2, fmt)
    want, off = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    xd = x.double()
    for e in range(w1.shape[0]):
        part = (weights.double() * (ids == e)).sum(1, keepdim=True)
        u, size = xd @ a1[e].t(), (dim + 8) * 2.0 ** -24 * (xd.abs() @ a1[e].abs().t())
        f = parts(act, u[:, :hidden])[0]
        a = f * u[:, hidden:]
        da = 1.13 * size[:, :hidden] * u[:, hidden:].abs() + f.abs() * size[:, hidden:] + 2.0 ** -15 * a.abs()
        da = da + (2.0 ** -8 + (hidden + ids.numel() + 16) * 2.0 ** -24) * a.abs()
        want += part * (a @ a2[e].t())
        off += part.abs() * (1.01 * da @ a2[e].abs().t())
    assert bool(torch.isfinite(y).all())
    bad = ((y.double() - want).abs() > 2.0 ** -8 * want.abs() + off + 1e-30)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values"


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k", [
    (1, 16, 16, 1, 1), (1, 128, 128, 8, 2), (1, 4096, 512, 16, 8), (2, 144, 80, 5, 5), (13, 528, 208, 40, 6), (16, 512, 256, 4, 2),
    (17, 512, 256, 4, 2), (33, 272, 400, 3, 1), (64, 384, 256, 8, 8), (64, 1040, 128, 1, 1), (64, 256, 144, 64, 16), (5, 32, 2064, 7, 3),
    (64, 128, 128, 130, 8), (3, 8208, 16, 4, 2),
    (64, 4112, 144, 20, 16)])
@pytest.mark.parametrize("fmt", [qf8.E4M3, qf8.E5M2])
def test_layer(tokens, dim, hidden, experts, top_k, fmt):
    act = ACTS[tokens % 2]
    args = made(tokens, dim, hidden, experts, top_k, fmt, seed=tokens + dim)
    y = qf8.expert_layer_tokens(*args, fmt, act=act)
    check(y, *args, fmt, act)
    assert torch.equal(y, qf8.expert_layer_tokens(*args, fmt, act=act))


def test_choices_of_any_kind():
    """Experts outside the layer, the same expert twice, tokens without any, all tokens on one expert."""
    ids = torch.tensor([[0, 0, 0], [1, 5, 1], [-1, 6, 99], [2, -1, 2], [-5, 1 << 30, -(1 << 31)], [5, 4, 3]], dtype=torch.int32, device="cuda")
    args = made(6, 256, 192, 6, 3, qf8.E4M3, seed=1, ids=ids)
    y = qf8.expert_layer_tokens(*args, qf8.E4M3)
    check(y, *args, qf8.E4M3, qf8.ACT_SILU)
    assert bool((y[2] == 0).all()) and bool((y[4] == 0).all())
    for counts in ([64], [33, 31], [32, 16, 16], [17, 47], [1, 2, 3, 40, 18]):       # pieces of one and two sixteens, and second pieces
        ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])[torch.randperm(sum(counts))].cuda()[:, None].contiguous()
        args = made(sum(counts), 272, 400, 6, 1, qf8.E4M3, seed=sum(counts), ids=ids)
        check(qf8.expert_layer_tokens(*args, qf8.E4M3), *args, qf8.E4M3, qf8.ACT_SILU)
    for expert in (0, 5, 7):
        ids = torch.full((40, 2), expert, dtype=torch.int32, device="cuda")
        args = made(40, 256, 192, 6, 2, qf8.E4M3, seed=2, ids=ids)
        check(qf8.expert_layer_tokens(*args, qf8.E4M3), *args, qf8.E4M3, qf8.ACT_SILU)


def test_the_same_bits_again():
    """Experts with several pieces of tokens, whose choices lie far apart: the order of the sums is the same in every run."""
    for top_k, experts in ((16, 20), (8, 8), (3, 3)):
        args = made(64, 512, 272, experts, top_k, qf8.E4M3, seed=experts)
        want = qf8.expert_layer_tokens(*args, qf8.E4M3)
        for _ in range(20):
            assert torch.equal(want, qf8.expert_layer_tokens(*args, qf8.E4M3))


def test_most_experts():
    ids = (torch.arange(64 * 16, device="cuda", dtype=torch.int32) % 1024).view(64, 16).contiguous()
    args = made(64, 128, 32, 1024, 16, qf8.E4M3, seed=3, ids=ids)
    check(qf8.expert_layer_tokens(*args, qf8.E4M3), *args, qf8.E4M3, qf8.ACT_SILU)


def test_a_token_does_not_touch_another():
    """Inf and NaN of one token stay in its row; a NaN weight of one expert in the rows that chose it."""
    x, w1, s1, w2, s2, ids, weights = made(20, 256, 128, 4, 2, qf8.E4M3, seed=4)
    want = qf8.expert_layer_tokens(x, w1, s1, w2, s2, ids, weights, qf8.E4M3)
    bad = x.clone()
    bad[3, 7], bad[11, 0] = float("inf"), float("nan")
    got = qf8.expert_layer_tokens(bad, w1, s1, w2, s2, ids, weights, qf8.E4M3)
    rows = torch.arange(20, device="cuda")
    others = (rows != 3) & (rows != 11)
    assert torch.equal(got[others], want[others]) and bool(got[11].isnan().all())
    w2 = w2.clone()
    w2[1, 5, 9] = 0x7F
    got = qf8.expert_layer_tokens(x, w1, s1, w2, s2, ids, weights, qf8.E4M3)
    chose = (ids == 1).any(1)
    assert torch.equal(got[~chose], want[~chose]) and torch.equal(got[:, :5], want[:, :5]) and bool(got[chose, 5].isnan().all())


def test_sizes_of_nothing_and_refusals():
    args = list(made(4, 256, 128, 4, 2, qf8.E4M3))
    empty = [args[0][:0], *args[1:5], args[5][:0], args[6][:0]]
    assert qf8.expert_layer_tokens(*empty, qf8.E4M3).shape == (0, 256)
    z = torch.zeros
    none = qf8.expert_layer_tokens(args[0], z(4, 0, 256, dtype=torch.uint8, device="cuda"), z(4, 0, 2, device="cuda"),
                                   z(4, 256, 0, dtype=torch.uint8, device="cuda"), z(4, 2, 0, device="cuda"), *args[5:], qf8.E4M3)
    assert bool((none == 0).all())
    with pytest.raises(TypeError):
        qf8.expert_layer_tokens(args[0].float(), *args[1:], qf8.E4M3)
    with pytest.raises(ValueError):
        qf8.expert_layer_tokens(*args[:3], args[3][:, :, :64].contiguous(), *args[4:], qf8.E4M3)
    with pytest.raises(ValueError):
        qf8.expert_layer_tokens(*args[:5], args[5][:3], args[6], qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.expert_layer_tokens(*args[:5], args[5].long(), args[6], qf8.E4M3)
    with pytest.raises(qf8.QF8Error):
        qf8.expert_layer_tokens(*args, qf8.E4M3, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    many = made(65, 128, 64, 4, 2, qf8.E4M3)
    with pytest.raises(qf8.QF8Error):
        qf8.expert_layer_tokens(*many, qf8.E4M3)
