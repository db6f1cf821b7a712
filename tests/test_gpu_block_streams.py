"""The operators around the expert layer on streams: each call on the given one and not on the current one, two at once with inputs and
workspaces of their own, and two captured graphs."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_expert_block import example

pytestmark = pytest.mark.gpu


def calls(seed):
    """Each call with all its inputs made beforehand; takes the stream."""
    x, residual, norm, router, w1, w2, dout, dh = example.inputs(40, 512, 256, 8, seed=seed)
    block = example.ExpertBlock(norm, router, w1, w2, 2)
    ids, weights = qf8.route_experts(x @ router.t(), 2)
    n = qf8.rms_norm_quantize(x, norm, None, want_rstd=True)
    grads, half = [dout, dh.float(), norm], dout[:, :256].contiguous()
    place = [torch.empty_like(g) for g in grads]
    return {
        "norm": lambda s: list(qf8.rms_norm_quantize(x, norm, qf8.E4M3, residual=residual, want_y=True, want_rstd=True, stream=s)),
        "norm_backward": lambda s: list(qf8.rms_norm_backward(dout, x, n.rstd, norm, dres=dh, stream=s)),
        "gate": lambda s: list(qf8.gated_act_quantize(x, qf8.E4M3, want_y=True, stream=s)),
        "gate_backward": lambda s: list(qf8.gated_act_backward(half, x, qf8.E5M2, want_dx=True, stream=s)),
        "layer": lambda s: [qf8.expert_layer_tokens(x, *block.w1, *block.w2, ids, weights, qf8.E4M3, stream=s)],
        "clip": lambda s: [qf8.clip_grads(grads, 1.0, out=place, stream=s), *place],
        "grad_norm": lambda s: [qf8.grad_norm(grads, stream=s)],
    }


NAMES = ["norm", "norm_backward", "gate", "gate_backward", "layer", "clip", "grad_norm"]


def two_streams():
    """A pair that runs side by side: the process's streams share a few hardware queues, and two of one queue run one after the other."""
    busy, done, word = torch.cuda.Stream(), torch.cuda.Event(), torch.zeros(1, device="cuda")
    for side in [torch.cuda.Stream() for _ in range(8)]:
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(20_000_000)
            done.record()
        with torch.cuda.stream(side):
            word.add_(1)
        side.synchronize()
        if not done.query():
            torch.cuda.synchronize()
            return busy, side
    pytest.skip("no two streams run side by side here")


@pytest.mark.parametrize("name", NAMES)
def test_on_the_given_stream(name):
    """While the current stream is busy, the call on another one ends: its results are there before the current stream's are. The
    memory that it writes holds zeros before."""
    call = calls(7)[name]
    want = [t.cpu() for t in call(None)]
    busy, side = two_streams()
    with torch.cuda.stream(side):
        for t in call(side):
            t.zero_()
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(100_000_000)
        done.record()
        got = call(side)
    with torch.cuda.stream(side):
        got = [t.cpu() for t in got]
    assert not done.query(), "the busy stream ended before the call was looked at"
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_two_at_once(name):
    """Different inputs on two streams, many calls in flight on both."""
    pair = [calls(seed)[name] for seed in (7, 8)]
    want = [[t.clone() for t in call(None)] for call in pair]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append((i, [t.clone() for t in pair[i](None)]))
    torch.cuda.synchronize()
    for i, tensors in got:
        assert all(torch.equal(g, w) for g, w in zip(tensors, want[i]))


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs(name):
    """Captured one after the other and replayed on two streams at once, with eager calls between."""
    pair = [calls(seed)[name] for seed in (9, 10)]
    want = [[t.clone() for t in call(None)] for call in pair]
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph, call in zip(graphs, pair):
        with torch.cuda.graph(graph):
            held.append(call(None))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for tensors in held:
            for t in tensors:
                t.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(g, w) for g, w in zip(held[i], want[i]))
            assert all(torch.equal(g, w) for g, w in zip(pair[i](None), want[i]))
