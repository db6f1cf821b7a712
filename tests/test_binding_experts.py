"""What the binding refuses before the library is called (CPU). Stand-ins for device tensors show shape, type,
layout and device as torch's do; the library is replaced, so that nothing is launched whatever is refused."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8


class Device:
    """A tensor on a device, as far as the binding looks at one."""

    def __init__(self, *shape, dtype=torch.float32, device=0, contiguous=True):
        self.shape, self.dtype, self.is_cuda, self.device_index, self.whole = torch.Size(shape), dtype, True, device, contiguous

    def is_contiguous(self):
        return self.whole

    def get_device(self):
        return self.device_index

    @property
    def device(self):
        return torch.device("cuda", self.device_index)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return 0x10000

    def new_empty(self, *shape, dtype=None):
        return Device(*shape, dtype=dtype or self.dtype, device=self.device_index)


@pytest.fixture
def calls(monkeypatch):
    """Names of the library's entry points that were called."""
    made = []
    real = qf8._load()

    class Library:
        def __getattr__(self, name):
            if name.endswith("_rows") or name.endswith("_bytes"):
                return getattr(real, name)
            return lambda *args: made.append(name) or 0
    monkeypatch.setattr(qf8, "_load", lambda: Library())
    monkeypatch.setattr(qf8, "_stream_of", lambda stream, t: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, Device), raising=True)
    return made


def u8(*s, **kw):
    return Device(*s, dtype=torch.uint8, **kw)


def i32(*s, **kw):
    return Device(*s, dtype=torch.int32, **kw)


def f32(*s, **kw):
    return Device(*s, **kw)


def product(ws):
    return lambda: qf8.matmul_block(u8(8, 65536), f32(8, 512), u8(128, 65536), f32(1, 512), qf8.E4M3, qf8.E4M3, ws=ws)


def order(ws):
    return lambda: qf8.order_experts(i32(4096, 8), 64, ws=ws)


@pytest.mark.parametrize("call", [product, order])
def test_workspace(call, calls):
    big = 1 << 24
    with pytest.raises(TypeError, match="ws"):
        call(torch.zeros(big, dtype=torch.uint8))()                                      # host memory
    with pytest.raises(TypeError, match="ws"):
        call(0x10000)()
    with pytest.raises(ValueError, match="ws"):
        call(u8(big, contiguous=False))()                                                # its span is not its size
    assert calls == []
    call(u8(big))()
    call(Device(4, big // 16, dtype=torch.float32))()                                    # any type and shape
    assert len(calls) == 2


def given(name):
    """Arguments by name of one right call, all on device 0."""
    i = dict(dtype=torch.int32)
    return {
        "matmul_block": dict(a=u8(8, 256), sa=f32(8, 2), b=u8(128, 256), sb=f32(1, 2), out=f32(8, 128), ws=u8(1 << 20),
                             fmt_a=0, fmt_b=0, out_dtype=torch.float32),
        "matmul_block_experts": dict(a=u8(8, 256), sa=f32(8, 2), b=u8(4, 128, 256), sb=f32(4, 1, 2), offsets=Device(5, **i),
                                     rows=Device(12, **i), out=f32(12, 128), fmt_a=0, fmt_b=0, out_dtype=torch.float32),
        "matmul_block_experts_wgrad": dict(at=u8(64, 256), sat=f32(64, 2), bt=u8(32, 256), sbt=f32(32, 2),
                                           offsets=Device(5, **i), out=f32(4, 64, 32), fmt_a=0, fmt_b=0),
        "route_experts": dict(logits=f32(6, 16), bias=f32(16), ids=Device(6, 2, **i), weights=f32(6, 2), top_k=2),
        "route_experts_backward": dict(logits=f32(6, 16), ids=Device(6, 2, **i), dweights=f32(6, 2), dlogits=f32(6, 16)),
        "order_experts": dict(ids=Device(6, 2, **i), offsets=Device(17, **i), rows=Device(12, **i), slots=Device(6, 2, **i),
                              ws=u8(1 << 20), experts=16),
        "combine_experts": dict(x=f32(12, 8), weights=f32(6, 2), slots=Device(6, 2, **i), y=f32(6, 8)),
        "combine_experts_backward": dict(x=f32(12, 8), dy=f32(6, 8), weights=f32(6, 2), slots=Device(6, 2, **i),
                                         rows=Device(12, **i), dx=f32(12, 8), dweights=f32(6, 2)),
    }[name]


@pytest.mark.parametrize("name", [n for n in qf8.__all__ if n.startswith(("matmul", "route", "order", "combine"))])
def test_one_device(name, calls):
    """Each tensor in its turn on another device than the others."""
    args = given(name)
    getattr(qf8, name)(**args)
    assert calls == [name]
    for which, t in args.items():
        if isinstance(t, Device):
            t.device_index = 1
            with pytest.raises(ValueError, match="one device"):
                getattr(qf8, name)(**args)
            t.device_index = 0
    assert calls == [name]
    none = {k: None for k in ("rows", "bias", "ws") if k in args and (k != "rows" or name == "matmul_block_experts")}
    if name == "matmul_block_experts":
        none.update(a=u8(12, 256), sa=f32(12, 2))
    getattr(qf8, name)(**{**args, **none})                  # what may be left out
    assert calls == [name, name]
