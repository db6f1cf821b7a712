"""stream= of every call of the products and the expert layer: outputs come from that stream's memory. A block that
the current stream has freed, but still has work pending on, is not taken."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8
from test_gpu_matmul import codes, operands, scales

pytestmark = pytest.mark.gpu


def calls():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(32)
    counts = torch.tensor([0, 128, 128, 384], dtype=torch.int32, device="cuda")
    a, sa = codes(gen, (384, 256), "e4m3"), scales(gen, (384, 2), False)
    b, sb, _ = operands(gen, "nk", 512, 256, "e4m3", False)
    b, sb = torch.stack([b] * 3), torch.stack([sb] * 3)
    at, sat = codes(gen, (256, 384), "e5m2"), scales(gen, (256, 3), False)
    bt, sbt = codes(gen, (512, 384), "e4m3"), scales(gen, (512, 3), False)
    logits = torch.randn(3000, 64, generator=gen, device="cuda")
    bias = torch.zeros(64, device="cuda")
    ids, w = qf8.route_experts(logits, 4)
    offsets, rows, slots = qf8.order_experts(ids, 64, align=16)
    x = torch.randn(rows.numel(), 264, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(3000, 264, generator=gen, device="cuda").to(torch.bfloat16)
    return {
        "matmul_block_experts": lambda s: (qf8.matmul_block_experts(a, sa, b, sb, counts, 0, 0, stream=s),),
        "matmul_block_experts_wgrad": lambda s: (qf8.matmul_block_experts_wgrad(at, sat, bt, sbt, counts, 1, 0, stream=s),),
        "route_experts": lambda s: qf8.route_experts(logits, 4, bias=bias, stream=s),
        "route_experts_backward": lambda s: (qf8.route_experts_backward(logits, ids, w, stream=s),),
        "combine_experts_backward": lambda s: qf8.combine_experts_backward(dy, x, w, slots, rows, stream=s),
    }


@pytest.mark.parametrize("name", ["matmul_block_experts", "matmul_block_experts_wgrad", "route_experts",
                                  "route_experts_backward", "combine_experts_backward"])
def test_outputs_belong_to_the_given_stream(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    old = [torch.empty_like(t) for t in want for _ in range(4)]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    for t in old:
        t.fill_(7)
    del t, old
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(got, want))


def test_the_whole_layer_on_another_stream():
    """Every call on one stream, with the current one busy."""
    results = []
    for stream in (None, torch.cuda.Stream()):
        made = calls()
        torch.cuda.synchronize()
        if stream is not None:
            torch.cuda._sleep(20_000_000)
        out = [t for name in made for t in made[name](stream)]
        if stream is not None:
            stream.synchronize()
        torch.cuda.synchronize()
        results.append(out)
    assert all(torch.equal(g, t) for g, t in zip(*results))
