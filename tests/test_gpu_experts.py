"""The expert layer around its products: choice of experts, order of the rows, weighted sum, and
their gradients, against plain fp64 implementations."""
import math

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
SCORE = {"softmax": qf8.SCORE_SOFTMAX, "sigmoid": qf8.SCORE_SIGMOID}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def scores64(logits, score):
    """fp64 scores; what cannot be chosen (-Inf, NaN) is 0."""
    l = logits.double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.max(dim=1, keepdim=True)[0]
    e = torch.exp(l - torch.where(torch.isinf(top), 0.0, top))
    return e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)


def plain_route(logits, top_k, score, bias, groups, top_groups, renorm, scale):
    s = scores64(logits, score)
    t, e = s.shape
    if bias is None and groups == 1:
        choice = torch.where(torch.isnan(logits), -math.inf, logits).double()
    else:
        choice = s if bias is None else s + bias.double()
    choice = choice.cpu().tolist()
    ids = []
    size = e // groups
    for row in choice:
        open_ = set(range(groups))
        if groups > 1:
            worth = [sum(sorted(row[g * size:(g + 1) * size], reverse=True)[:2]) for g in range(groups)]
            open_ = set(sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups])
        cand = [i for i in range(e) if i // size in open_]
        ids.append(sorted(cand, key=lambda i: (-row[i], i))[:top_k])
    ids = torch.tensor(ids, dtype=torch.int64, device=logits.device)
    w = s.gather(1, ids)
    if renorm:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp_min(1e-300), 0.0)
    return ids, w * scale


def check_route(logits, top_k, score="softmax", bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    ids, w = qf8.route_experts(logits, top_k, score=SCORE[score], bias=bias, groups=groups, top_groups=top_groups,
                               renorm=renorm, scale=scale)
    torch.cuda.synchronize()
    want_ids, want_w = plain_route(logits, top_k, score, bias, groups, top_groups, renorm, scale)
    assert torch.equal(ids.long(), want_ids), torch.nonzero(ids.long() != want_ids)[:3].tolist()
    # fp64 all through, rounded once to fp32; fp64's own error is far below the slack
    assert bool(((w.double() - want_w).abs() <= want_w.abs() * (2.0 ** -24 * 1.01) + 1e-45).all())
    return ids, w


def random_logits(tokens, experts, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (2.0 * torch.randn(tokens, experts, generator=gen, device="cuda")).to(dtype), gen


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (3, 8, 2), (5, 60, 4), (64, 64, 8), (17, 100, 6), (33, 128, 1),
                                                  (9, 256, 8), (1030, 160, 6), (4, 512, 10), (3, 1000, 32), (2, 1024, 64)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(tokens, experts, top_k, dtype, score):
    x, gen = random_logits(tokens, experts, dtype, tokens + experts)
    bias = 0.1 * torch.randn(experts, generator=gen, device="cuda")
    for b in (None, bias):
        for renorm in (False, True):
            check_route(x, top_k, score, bias=b, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 4, 1, 4), (60, 3, 2, 8),
                                                             (128, 64, 8, 8), (32, 32, 5, 4), (1024, 16, 2, 16), (40, 5, 5, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups(experts, groups, top_groups, top_k, score):
    for dtype in (torch.bfloat16, torch.float32):
        x, gen = random_logits(37, experts, dtype, experts)
        bias = 0.1 * torch.randn(experts, generator=gen, device="cuda")
        check_route(x, top_k, score, groups=groups, top_groups=top_groups)
        check_route(x, top_k, score, bias=bias, groups=groups, top_groups=top_groups, renorm=False)


def test_route_ties_take_the_lowest_index():
    x = torch.zeros(5, 96, device="cuda")
    x[1, 70] = x[1, 10] = 1.0
    x[2] = -0.0
    x[2, ::2] = 0.0
    for score in ("softmax", "sigmoid"):
        ids, _ = check_route(x, 6, score)
        assert ids[0].tolist() == [0, 1, 2, 3, 4, 5] and ids[2].tolist() == [0, 1, 2, 3, 4, 5]
        assert ids[1].tolist() == [10, 70, 0, 1, 2, 3]
        check_route(x, 6, score, groups=4, top_groups=2)
        check_route(x, 6, score, bias=torch.zeros(96, device="cuda"))


def test_route_near_ties_need_fp64():
    """Scores that fp32 cannot tell apart are ordered by their fp64 values."""
    x = torch.zeros(4, 32, device="cuda")
    x[:, 20] = 2.0 ** -30
    bias = torch.full((32,), 0.25, device="cuda")
    for score in ("softmax", "sigmoid"):
        ids, _ = check_route(x, 3, score, bias=bias)
        assert ids[:, 0].tolist() == [20] * 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_rows(dtype, score):
    """-Inf and NaN logits, the type's lowest value, and rows with nothing left."""
    x, _ = random_logits(6, 72, dtype, 3)
    x[0, 5:] = -math.inf
    x[1] = -math.inf
    x[2, :70] = math.nan
    x[3, ::2] = torch.finfo(dtype).min
    x[4, 3] = torch.finfo(dtype).max
    for bias in (None, torch.linspace(-0.2, 0.2, 72, device="cuda")):
        for renorm in (False, True):
            ids, w = check_route(x, 8, score, bias=bias, renorm=renorm)
            assert bool(torch.isfinite(w).all())
    ids, w = qf8.route_experts(x, 8, score=SCORE[score])
    assert ids[1].tolist() == list(range(8)) and bool((w[1] == 0).all())
    d = qf8.route_experts_backward(x, ids, torch.ones_like(w), score=SCORE[score])
    assert bool(torch.isfinite(d.float()).all()) and bool((d[1] == 0).all())


def test_route_positive_infinity():
    x = torch.zeros(1, 16, device="cuda")
    x[0, 9] = math.inf
    ids, w = qf8.route_experts(x, 2)
    assert ids[0].tolist() == [9, 0] and w[0].tolist() == [1.0, 0.0]


def route_weights64(l, ids, score, renorm, scale):
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    w = s.gather(1, ids)
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (7, 8, 2), (33, 60, 4), (5, 256, 8), (3, 1000, 16), (1500, 64, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(tokens, experts, top_k, dtype, score, renorm):
    x, gen = random_logits(tokens, experts, dtype, experts)
    ids, w = qf8.route_experts(x, top_k, score=SCORE[score], renorm=renorm, scale=1.5)
    dw = torch.randn(tokens, top_k, generator=gen, device="cuda")
    got = qf8.route_experts_backward(x, ids, dw, score=SCORE[score], renorm=renorm, scale=1.5).double()
    l = x.double().cpu().requires_grad_()
    out = route_weights64(l, ids.long().cpu(), score, renorm, 1.5)
    (want,) = torch.autograd.grad(out, l, dw.double().cpu())
    want = want.to("cuda")
    # fp64 inside, one rounding; where the exact value is 0 (one chosen expert, or the others under
    # renormalisation) fp64 leaves about 2^-50 of the terms
    tol = want.abs() * HALF[dtype] * 1.01 + 2.0 ** -45 * dw.abs().double().max(dim=1, keepdim=True)[0]
    assert bool(((got - want).abs() <= tol).all())


def test_route_backward_against_differences():
    x, gen = random_logits(6, 24, torch.float32, 8)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = qf8.route_experts(x, 4, score=SCORE[score], renorm=renorm)
            dw = torch.randn(6, 4, generator=gen, device="cuda")
            got = qf8.route_experts_backward(x, ids, dw, score=SCORE[score], renorm=renorm).double()
            l, i, h = x.double(), ids.long(), 1e-4
            for e in range(24):
                up, dn = l.clone(), l.clone()
                up[:, e] += h
                dn[:, e] -= h
                f = lambda v: (route_weights64(v, i, score, renorm, 1.0) * dw.double()).sum(1)
                num = (f(up) - f(dn)) / (2 * h)
                # central differences: h^2 / 6 times a third derivative of at most 8 sum |dw|, and
                # fp64 cancellation of 2^-50 / h; then one fp32 rounding
                tol = h * h * 8 / 6 * dw.abs().double().sum(1) + 1e-11 + num.abs() * 2.0 ** -23
                assert bool(((got[:, e] - num).abs() <= tol).all()), (score, renorm, e)


def plain_order(ids, experts, align, nrows):
    t, k = ids.shape
    flat = ids.reshape(-1).tolist()
    offsets, rows, slots = [0], [-1] * nrows, [-1] * len(flat)
    for e in range(experts):
        at = offsets[-1]
        n = 0
        for i, v in enumerate(flat):
            if v == e:
                rows[at + n], slots[i] = i // k, at + n
                n += 1
        offsets.append(at + -(-n // align) * align)
    return offsets, rows, slots


@pytest.mark.parametrize("tokens,experts,top_k,align", [(1, 1, 1, 1), (1, 8, 2, 16), (64, 64, 8, 1), (511, 8, 8, 128), (100, 60, 6, 16),
                                                        (513, 16, 8, 1), (1000, 64, 6, 128), (3000, 33, 4, 7), (40, 1024, 64, 2),
                                                        (2048, 256, 8, 128), (9, 1000, 3, 1024)])
def test_order(tokens, experts, top_k, align):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    ids = torch.randint(0, experts, (tokens, top_k), generator=gen, device="cuda", dtype=torch.int32)
    ids[torch.rand(tokens, top_k, generator=gen, device="cuda") < 0.3] = experts // 2      # one popular expert
    n = tokens * top_k
    nrows = -(-(n + min(experts, n) * (align - 1)) // align) * align
    guard = torch.full((nrows + 64,), 12345, dtype=torch.int32, device="cuda")
    offsets, rows, slots = qf8.order_experts(ids, experts, align=align, rows=guard[:nrows])
    torch.cuda.synchronize()
    assert bool((guard[nrows:] == 12345).all())
    want = plain_order(ids.cpu(), experts, align, nrows)
    assert offsets.tolist() == want[0]
    assert rows.tolist() == want[1]
    assert slots.reshape(-1).tolist() == want[2]
    auto = qf8.order_experts(ids, experts, align=align)
    assert all(torch.equal(a, b) for a, b in zip(auto, (offsets, rows, slots)))


@pytest.mark.parametrize("tokens", [5, 3000])
def test_order_drops_ids_out_of_range(tokens):
    ids = torch.arange(tokens * 4, device="cuda", dtype=torch.int32).view(tokens, 4) % 10 - 1       # -1 .. 8
    offsets, rows, slots = qf8.order_experts(ids, 8, align=4)
    want = plain_order(ids.cpu(), 8, 4, rows.numel())
    assert offsets.tolist() == want[0] and rows.tolist() == want[1] and slots.reshape(-1).tolist() == want[2]


def test_order_no_tokens():
    offsets, rows, slots = qf8.order_experts(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 8, align=16)
    assert offsets.tolist() == [0] * 9 and rows.numel() == 0 and slots.shape == (0, 4)


def combine_case(tokens, experts, top_k, dim, dtype, align=1, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ids = torch.rand(tokens, experts, generator=gen, device="cuda").topk(top_k, 1)[1].to(torch.int32)
    offsets, rows, slots = qf8.order_experts(ids, experts, align=align)
    x = torch.randn(rows.numel(), dim, generator=gen, device="cuda").to(dtype)
    w = torch.randn(tokens, top_k, generator=gen, device="cuda")
    dy = torch.randn(tokens, dim, generator=gen, device="cuda").to(dtype)
    return x, w, slots, rows, dy


@pytest.mark.parametrize("tokens,experts,top_k,dim", [(1, 8, 1, 8), (5, 8, 2, 1), (64, 16, 8, 7168), (33, 8, 3, 130), (3, 32, 16, 333),
                                                      (2100, 8, 2, 264), (1, 64, 9, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine(tokens, experts, top_k, dim, dtype):
    print(f"combine {tokens} {experts} {top_k} {dim} {dtype}", flush=True)
    x, w, slots, rows, dy = combine_case(tokens, experts, top_k, dim, dtype, align=16, seed=dim)
    x[rows < 0] = math.nan                                   # padding rows are not read
    y = qf8.combine_experts(x, w, slots)
    dx, dw = qf8.combine_experts_backward(dy, x, w, slots, rows)
    torch.cuda.synchronize()
    xs = x.double()[slots.long().reshape(-1)].view(tokens, top_k, dim)
    terms = w.double()[:, :, None] * xs
    want = terms.sum(1)
    tol = want.abs() * HALF[dtype] * 1.01 + terms.abs().sum(1) * (top_k * 2.0 ** -24)
    assert bool(((y.double() - want).abs() <= tol).all())
    wdx = torch.zeros(rows.numel(), dim, dtype=torch.float64, device="cuda")
    wdx[slots.long().reshape(-1)] = (w.double()[:, :, None] * dy.double()[:, None, :]).reshape(-1, dim)
    # one product in fp32, one rounding to the type
    assert bool(((dx.double() - wdx).abs() <= wdx.abs() * (HALF[dtype] + 2.0 ** -24) * 1.01 + 1e-45).all())
    assert bool((dx[rows < 0] == 0).all())
    prod = dy.double()[:, None, :] * xs
    wdw = prod.sum(2)
    assert bool(((dw.double() - wdw).abs() <= prod.abs().sum(2) * ((dim + 8) * 2.0 ** -24)).all())


def test_combine_slots_out_of_range():
    x, w, slots, rows, dy = combine_case(12, 8, 4, 72, torch.float32)
    slots[3, 1] = -1
    slots[5, 0] = rows.numel()
    rows[int(slots[7, 2])] = -1
    y = qf8.combine_experts(x, w, slots)
    dx, dw = qf8.combine_experts_backward(dy, x, w, slots, rows)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < rows.numel())
    xs = torch.where(ok[:, :, None], x.double()[slots.clamp(0, rows.numel() - 1).long()], 0.0)
    terms = w.double()[:, :, None] * xs
    assert bool(((y.double() - terms.sum(1)).abs() <= terms.abs().sum(1) * 2.0 ** -21).all())
    assert dw[3, 1].item() == 0 and dw[5, 0].item() == 0


def test_combine_same_bits_again():
    x, w, slots, rows, dy = combine_case(50, 16, 8, 1000, torch.bfloat16)
    a = qf8.combine_experts_backward(dy, x, w, slots, rows)
    b = qf8.combine_experts_backward(dy, x, w, slots, rows)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tokens", [16, 1500])
def test_graph_replays_the_layer(tokens):
    """Choice, order and sum captured together; replays follow new logits in place."""
    x, gen = random_logits(tokens, 64, torch.float32, 1)
    rows_in = torch.randn(-(-(tokens * 4 + 64 * 15) // 16) * 16, 256, generator=gen, device="cuda").to(torch.bfloat16)

    def layer():
        ids, w = qf8.route_experts(x, 4, score=qf8.SCORE_SIGMOID)
        offsets, rows, slots = qf8.order_experts(ids, 64, align=16)
        return ids, w, offsets, rows, slots, qf8.combine_experts(rows_in, w, slots)

    layer()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer()
    for i in range(4):
        x.copy_(torch.randn(tokens, 64, generator=gen, device="cuda"))
        want = layer()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("tokens,experts,top_k", [(4097, 1, 1), (4098, 8, 8), (4099, 60, 4), (4097, 64, 16), (4101, 100, 6),
                                                  (4103, 128, 8), (8193, 129, 3), (8194, 256, 8), (8193, 250, 17)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_many_tokens(tokens, experts, top_k, dtype):
    """Four tokens share a wave: token counts that leave rows of lanes empty, and masks and ties in some."""
    x, gen = random_logits(tokens, experts, dtype, tokens + experts)
    x[5] = float("-inf")
    x[6] = 1.25
    x[tokens - 1, experts // 2:] = float("-inf")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            check_route(x, top_k, score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("tokens,experts,top_k", [(2051, 8, 2), (2050, 60, 4), (2049, 128, 8), (3001, 256, 16), (2053, 250, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_backward_many_tokens(tokens, experts, top_k, dtype):
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            test_route_backward(tokens, experts, top_k, dtype, score, renorm)


def test_route_backward_many_tokens_masked():
    """Masked rows and ids outside the experts, among many tokens: the same values as a few at a time."""
    x, gen = random_logits(2500, 96, torch.float32, 12)
    x[7] = float("-inf")
    x[11, 3:] = float("-inf")
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, _ = qf8.route_experts(x, 5, score=SCORE[score], renorm=renorm)
            ids[13, 2], ids[14, 0] = -1, 96
            dw = torch.randn(2500, 5, generator=gen, device="cuda")
            got = qf8.route_experts_backward(x, ids, dw, score=SCORE[score], renorm=renorm)
            few = torch.cat([qf8.route_experts_backward(x[i:i + 500].contiguous(), ids[i:i + 500].contiguous(),
                                                        dw[i:i + 500].contiguous(), score=SCORE[score], renorm=renorm)
                             for i in range(0, 2500, 500)])
            # sums of at most 96 terms in fp64, in another order, then one rounding each
            tol = few.abs().double() * 2.0 ** -23 + 2.0 ** -45 * dw.abs().double().max(dim=1, keepdim=True)[0]
            assert bool(((got.double() - few.double()).abs() <= tol).all()) and bool(torch.isfinite(got).all())
