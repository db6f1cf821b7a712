"""The FP8 expert layer of examples/expert_layer.py against the same layer without quantization.

Tolerances, relative to the norm: the half steps of the roundings on the way, E4M3 2^-4 and E5M2 2^-3
each. y: x, w1, act, w2. dx: that of the choice's weights (y's) and of dv, w2, du, w1. dw2: dv twice
(re-grouped once), act twice and what act holds of x and w1; dw1: du twice and what it holds of dv
and w2, x twice."""
import importlib.util
import os

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
_spec = importlib.util.spec_from_file_location(
    "expert_layer", os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py"))
layer_example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(layer_example)
E4, E5 = 2.0 ** -4, 2.0 ** -3


@pytest.mark.parametrize("tokens,dim,hidden,experts,top_k", [(300, 512, 256, 8, 2), (65, 384, 272, 16, 4), (1, 256, 128, 4, 1)])
def test_training_step(tokens, dim, hidden, experts, top_k):
    print(f"expert layer {tokens} {dim} {hidden} {experts} {top_k}", flush=True)
    x, router, w1, w2, dy = layer_example.inputs(tokens, dim, hidden, experts)
    layer = layer_example.ExpertLayer(router, w1, w2, top_k)
    y, saved = layer.forward(x, training=True)
    got = (y, *layer.backward(dy, saved))
    want = layer_example.reference(x, router, w1, w2, saved[2], dy)
    tol = {"y": 4 * E4, "dx": 4 * E4 + 2 * E5 + 2 * E4, "dw1": 2 * E5 + E5 + E4 + 2 * E4, "dw2": 2 * E5 + 2 * E4 + 2 * E4}
    for name, g, w in zip(("y", "dx", "drouter", "dw1", "dw2"), got, want):
        assert g.shape == w.shape and bool(torch.isfinite(g).all())
        if name in tol:
            diff = float((g.float() - w).norm())
            assert diff <= tol[name] * float(w.norm()), f"{name}: {diff / float(w.norm()):.3f} of the norm"


def test_decoding_matches_training_rows():
    """The same tokens with and without padded experts: the same products, row by row."""
    x, router, w1, w2, _ = layer_example.inputs(48, 512, 256, 8, seed=3)
    layer = layer_example.ExpertLayer(router, w1, w2, 2, score=qf8.SCORE_SIGMOID, groups=4, top_groups=2, scale=2.5)
    a, sa = layer.forward(x)
    b, sb = layer.forward(x, training=True)
    assert bool((sa[2] == sb[2]).all())
    assert float((a.float() - b.float()).norm()) <= 2.0 ** -8 * 4 * float(b.float().norm())


def test_step_replays_in_a_graph():
    """Decoding captured once and replayed over new tokens gives the eager results."""
    x, router, w1, w2, _ = layer_example.inputs(64, 512, 256, 8, seed=5)
    layer = layer_example.ExpertLayer(router, w1, w2, 2)
    static = x.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = layer.forward(static)
    for seed in range(4):
        fresh = layer_example.inputs(64, 512, 256, 8, seed=10 + seed)[0]
        want = layer.forward(fresh)[0].clone()
        static.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
