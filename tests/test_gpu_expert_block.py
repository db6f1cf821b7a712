"""The block of examples/expert_block.py: norm, router, gated experts and clipping as they are used together, against
the same block without quantization; and its decoding step, captured and replayed.

Tolerances, relative to the norm: the half steps of the roundings on the way, E4M3 2^-4 and E5M2 2^-3 each. out: z, w1, the
activation, w2. dx: that of the choice's weights (out's) and of dv, w2, du, w1 and the forward's z, w1 in the gate's slope. dw2: dv
twice (re-grouped once), the activation twice and what it holds of z and w1; dw1: du twice and what it holds of dv, w2, z and w1, z
twice. dnorm as dx. In the decoding step only the weights are rounded to FP8."""
import importlib.util
import os

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
_spec = importlib.util.spec_from_file_location(
    "expert_block", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)
E4, E5 = 2.0 ** -4, 2.0 ** -3


def close(name, got, want, tol):
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), name
    diff = float((got.double() - want.double()).norm()) / float(want.double().norm())
    assert diff <= tol, f"{name}: {diff:.4f} of the norm, {tol:.4f} allowed"


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k,act", [
    (300, 512, 256, 8, 2, qf8.ACT_SILU), (65, 384, 128, 16, 4, qf8.ACT_GELU), (1, 256, 128, 4, 1, qf8.ACT_SILU)])
def test_training_step(tokens, dim, hidden, experts, top_k, act):
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(tokens, dim, hidden, experts)
    block = example.ExpertBlock(norm, router, w1, w2, top_k, act=act)
    out, h, saved = block.forward(x, residual)
    got = (out, h, *block.backward(dout, dh, saved))
    want = example.reference(x, residual, norm, router, w1, w2, saved[2], act, dout, dh)
    tol = {"out": 4 * E4, "h": 2.0 ** -8, "dx": 4 * E4 + 2 * E5 + 4 * E4, "dnorm": 4 * E4 + 2 * E5 + 4 * E4,
           "dw1": 3 * E5 + 6 * E4, "dw2": 2 * E5 + 4 * E4}
    for name, g, w in zip(("out", "h", "dx", "dnorm", "drouter", "dw1", "dw2"), got, (*want[:3], *want[4:])):
        if name in tol:
            close(name, g, w, tol[name])
        else:
            assert g.shape == w.shape and bool(torch.isfinite(g).all())
    keep = [g.clone() for g in got[3:]]
    norm_of = sum(float(g.double().square().sum()) for g in keep) ** 0.5
    *_, grads, total = block.train(x, residual, dout, dh, 0.25 * norm_of)
    assert abs(total.item() - norm_of) <= 2.0 ** -23 * norm_of
    for g, k in zip(grads, keep):
        assert float((g.double() - 0.25 * k.double()).norm()) <= 2.0 ** -7 * float(k.double().norm())


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k", [(1, 512, 256, 8, 2), (48, 384, 256, 8, 3), (64, 256, 128, 4, 4)])
def test_decoding_step(tokens, dim, hidden, experts, top_k):
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(tokens, dim, hidden, experts, seed=3)
    block = example.ExpertBlock(norm, router, w1, w2, top_k)
    out, h = block.decode(x, residual)
    y = qf8.rms_norm_quantize(x, norm, None, residual=residual).y
    ids = qf8.route_experts(y @ router.t(), top_k)[0]
    want = example.reference(x, residual, norm, router, w1, w2, ids, block.act, dout, dh)
    close("out", out, want[0], 2 * E4 + 2.0 ** -6)
    close("h", h, want[1], 2.0 ** -8)
    trained = block.forward(x, residual)
    assert torch.equal(trained[1], h)
    close("out of training", trained[0], want[0], 4 * E4)


def test_decoding_replays_in_a_graph():
    """Captured once and replayed over new tokens, with eager work and synchronizations between: the eager results."""
    x, residual, norm, router, w1, w2, *_ = example.inputs(24, 512, 256, 8, seed=5)
    block = example.ExpertBlock(norm, router, w1, w2, 2)
    sx, sr = x.clone(), residual.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.decode(sx, sr)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = block.decode(sx, sr)
    for seed in range(4):
        fresh = example.inputs(24, 512, 256, 8, seed=10 + seed)[:2]
        want, hwant = (t.clone() for t in block.decode(*fresh))
        sx.copy_(fresh[0])
        sr.copy_(fresh[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h, hwant)


def calls():
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(40, 512, 256, 8, seed=7)
    block = example.ExpertBlock(norm, router, w1, w2, 2)
    ids, weights = qf8.route_experts(x @ router.t(), 2)
    n = qf8.rms_norm_quantize(x, norm, None, want_rstd=True)
    grads = [dout, dh.float(), norm]
    return {
        "norm": lambda s: [t for t in qf8.rms_norm_quantize(x, norm, qf8.E4M3, residual=residual, want_y=True, want_rstd=True, stream=s)],
        "norm_backward": lambda s: list(qf8.rms_norm_backward(dout, x, n.rstd, norm, dres=dh, stream=s)),
        "gate": lambda s: list(qf8.gated_act_quantize(x, qf8.E4M3, want_y=True, stream=s)),
        "gate_backward": lambda s: list(qf8.gated_act_backward(dout[:, :256].contiguous(), x, qf8.E5M2, want_dx=True, stream=s)),
        "layer": lambda s: [qf8.expert_layer_tokens(x, *block.w1, *block.w2, ids, weights, qf8.E4M3, stream=s)],
        "clip": lambda s: [t for o in [[torch.empty_like(g) for g in grads]] for t in (qf8.clip_grads(grads, 1.0, out=o, stream=s), *o)],
        "grad_norm": lambda s: [qf8.grad_norm(grads, stream=s)],
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "gate", "gate_backward", "layer", "clip", "grad_norm"])
def test_each_call_in_a_graph_and_on_a_stream(name):
    """The same bits eagerly, on another stream beside a busy one, and in every replay of a graph."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    if name not in ("clip", "gate_backward"):                # those make tensors on the current stream here
        torch.cuda._sleep(20_000_000)
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(None)
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(held, want))
        assert all(torch.equal(g, w) for g, w in zip(call(None), want))
