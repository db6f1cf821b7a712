"""The training step of examples/expert_layer.py, step by step against fp64 products of the same codes.

Up to dv every step starts from what the layer itself saved, so only the step's own rounding is between the two.
The gradient of the activation is BF16 and quantized again: half a BF16 step moves a value across a border of
E5M2 (step 2^-2) once in 2^6, by 2^-2 of it, which is 2^-5 of the norm, once more where codes are re-grouped.
Bounds, of the norm: dw2 its fp32 sums (2^-16); dw1 two such moves and dx one, beside the BF16 roundings on the
way (2^-8 each), in quadrature, since the roundings are independent of each other; the router's gradient the BF16
roundings of dlogits and of its product. CPU: leaving out a term, or a slope of the activation, exceeds them."""
import importlib.util
import math
import os

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

_spec = importlib.util.spec_from_file_location(
    "expert_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py"))
layer_example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(layer_example)

MOVE, BF16 = 2.0 ** -5, 2.0 ** -8
BOUND = {"y": math.hypot(BF16, BF16), "dw2": 2.0 ** -16, "dw1": math.hypot(MOVE, MOVE, BF16),
         "dx": math.hypot(MOVE, BF16, BF16, BF16, BF16), "drouter": math.hypot(BF16, BF16)}
DT = {qf8.E4M3: torch.float8_e4m3fn, qf8.E5M2: torch.float8_e5m2}


def values(codes, fmt, block_rows=1):
    q, s = codes
    full = s.double().repeat_interleave(block_rows, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.view(DT[fmt]).double() / full


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def by_expert(a, weights, offsets, transposed):
    """Rows of every expert times its weight (fp64)."""
    y = torch.zeros(a.shape[0], weights[0].shape[1 if transposed else 0], dtype=torch.float64, device=a.device)
    for e, w in enumerate(weights):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi] = torch.matmul(a[lo:hi], w if transposed else w.t().contiguous())
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k", [(300, 512, 256, 8, 2), (65, 384, 272, 16, 4), (33, 256, 128, 4, 1)])
def test_training_step(tokens, dim, hidden, experts, top_k):
    print(f"expert layer steps {tokens} {dim} {hidden} {experts} {top_k}", flush=True)
    x, router, w1, w2, dy = layer_example.inputs(tokens, dim, hidden, experts, seed=tokens)
    layer = layer_example.ExpertLayer(router, w1, w2, top_k)
    y, saved = layer.forward(x, training=True)
    dx, drouter, dw1, dw2 = layer.backward(dy, saved)
    _, logits, ids, weights, offsets, rows, slots, u, act, v = saved
    torch.cuda.synchronize()
    o, keep = offsets.tolist(), rows >= 0
    token = rows.clamp(min=0).long()
    flat = slots.long().reshape(-1)
    v1 = [values((layer.w1[0][e], layer.w1[1][e]), qf8.E4M3, 128) for e in range(experts)]
    v2 = [values((layer.w2[0][e], layer.w2[1][e]), qf8.E4M3, 128) for e in range(experts)]

    # forward
    xq = values(layer_example._groups(x, qf8.E4M3), qf8.E4M3)
    xr = torch.where(keep[:, None], xq[token], 0.0)
    assert off(u, by_expert(xr, v1, o, False)) <= BF16
    assert off(v, by_expert(values(act, qf8.E4M3), v2, o, False)) <= BF16
    want_y = (weights.double()[:, :, None] * v.double()[flat].view(tokens, top_k, dim)).sum(1)
    assert off(y, want_y) <= BOUND["y"]

    # backward: dv is weights * dy, rounded once
    dv = torch.zeros(rows.numel(), dim, dtype=torch.bfloat16, device="cuda")
    dv[flat] = (weights[:, :, None] * dy.float()[:, None, :]).to(torch.bfloat16).reshape(-1, dim)
    dvq = layer_example._groups(dv, qf8.E5M2)
    regroup = lambda q, fmt: values(qf8.requantize_1x128_to_128x1(*q, fmt, fmt), fmt)
    dvt, actt = regroup(dvq, qf8.E5M2), regroup(act, qf8.E4M3)
    want = torch.stack([torch.matmul(dvt[:, o[e]:o[e + 1]], actt[:, o[e]:o[e + 1]].t().contiguous()) for e in range(experts)])
    assert off(dw2, want) <= BOUND["dw2"]

    dact = by_expert(values(dvq, qf8.E5M2), v2, o, True)
    sig = torch.sigmoid(u.double())
    du = (dact * (sig * (1 + u.double() * (1 - sig)))).to(torch.bfloat16)
    duq = layer_example._groups(du, qf8.E5M2)
    xt = regroup(layer_example._groups(torch.where(keep[:, None], x[token], 0), qf8.E4M3), qf8.E4M3)
    dut = regroup(duq, qf8.E5M2)
    want = torch.stack([torch.matmul(dut[:, o[e]:o[e + 1]], xt[:, o[e]:o[e + 1]].t().contiguous()) for e in range(experts)])
    assert off(dw1, want) <= BOUND["dw1"]

    dxr = by_expert(values(duq, qf8.E5M2), v1, o, True)
    dweights = (dy.double()[:, None, :] * v.double()[flat].view(tokens, top_k, dim)).sum(2)
    p = torch.softmax(logits.double(), 1).gather(1, ids.long())
    w = p / p.sum(1, keepdim=True)
    dlogits = torch.zeros(tokens, experts, dtype=torch.float64, device="cuda")
    dlogits.scatter_(1, ids.long(), w * (dweights - (dweights * w).sum(1, keepdim=True)))
    of_router = torch.matmul(dlogits, router.double())
    of_experts = dxr[flat].view(tokens, top_k, dim).sum(1)
    assert off(dx, of_experts + of_router) <= BOUND["dx"]
    want = torch.matmul(dlogits.t().contiguous(), x.double())
    if top_k > 1:
        assert off(drouter, want) <= BOUND["drouter"]
        # the router's share alone: what is left of dx without the experts' share
        bound = BOUND["dx"] * float((of_experts + of_router).norm() / of_router.norm())
        assert bound < 0.5 and off(dx.double() - of_experts, of_router) <= bound
    else:
        assert bool((drouter == 0).all())                    # one chosen expert: its weight is 1


def test_a_missing_term_exceeds_the_bounds():
    """The same layer on the CPU in fp64, with one mistake at a time."""
    tokens, dim, hidden, experts, top_k = 300, 512, 256, 8, 2
    gen = torch.Generator()
    gen.manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    x, router, dy = normal(tokens, dim), normal(experts, dim) * dim ** -0.5, normal(tokens, dim)
    w1, w2 = normal(experts, hidden, dim) * dim ** -0.5, normal(experts, dim, hidden) * hidden ** -0.5
    ids = torch.topk(x @ router.t(), top_k, dim=1)[1]

    def gradients(mistake):
        p = torch.softmax(x @ router.t(), 1).gather(1, ids)
        w = p / p.sum(1, keepdim=True)
        y, dx = torch.zeros(tokens, dim, dtype=torch.float64), torch.zeros(tokens, dim, dtype=torch.float64)
        dw1, dw2, dlogits = torch.zeros_like(w1), torch.zeros_like(w2), torch.zeros(tokens, experts, dtype=torch.float64)
        dweights = torch.zeros(tokens, top_k, dtype=torch.float64)
        for e in range(experts):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            u = x[t] @ w1[e].t()
            sig = torch.sigmoid(u)
            act = u * sig
            v = act @ w2[e].t()
            y[t] += w[t, j][:, None] * v
            dweights[t, j] = (dy[t] * v).sum(1)
            dv = dy[t] if mistake == "weights of dv" else w[t, j][:, None] * dy[t]
            dw2[e] = dv.t() @ act
            slope = {"slope": sig, "half of the slope": sig * (1 + u)}.get(mistake, sig * (1 + u * (1 - sig)))
            du = (dv @ w2[e]) * slope
            dw1[e] = du.t() @ x[t]
            dx[t] += du @ w1[e]
        mean = 0.0 if mistake == "renormalisation" else (dweights * w).sum(1, keepdim=True)
        dlogits.scatter_(1, ids, w * (dweights - mean))
        if mistake != "router's share":
            dx = dx + dlogits @ router
        return {"y": y, "dx": dx, "drouter": dlogits.t() @ x, "dw1": dw1, "dw2": dw2}

    right = gradients(None)
    for mistake, seen in (("weights of dv", ("dx", "dw1", "dw2")), ("slope", ("dx", "dw1")), ("half of the slope", ("dx", "dw1")),
                          ("renormalisation", ("dx", "drouter")), ("router's share", ("dx",))):
        wrong = gradients(mistake)
        for name in seen:
            assert off(wrong[name], right[name]) > 2 * BOUND[name], (mistake, name)
