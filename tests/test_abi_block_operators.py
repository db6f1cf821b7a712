"""Refusals of the norm, the gated activation, the expert layer for a few tokens and the clipping of gradients (CPU:
nothing is launched)."""
import ctypes

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

OK, NULL, ENUM, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4, -5
F = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
UNEVEN = ctypes.c_void_p(0x10002)
INF = float("inf")


def lib():
    return qf8._load()


def norm(x=F, dt=0, r=F, rdt=0, w=F, wdt=0, rows=4, cols=256, eps=1e-6, fmt=0, flags=0, q=F, s=F, h=F, y=None, rstd=None, nf=None):
    return lib().rms_norm_quantize(x, dt, r, rdt, w, wdt, rows, cols, eps, fmt, flags, q, s, h, y, rstd, nf, None)


def test_norm_refusals():
    assert norm(dt=2) == ENUM and norm(rdt=-1) == ENUM and norm(wdt=3) == ENUM and norm(fmt=2) == ENUM and norm(flags=2) == ENUM
    assert norm(flags=16) == ENUM
    assert norm(rows=-1) == SHAPE and norm(cols=-8) == SHAPE and norm(cols=260) == SHAPE and norm(cols=16392) == SHAPE
    assert norm(eps=0.0) == SHAPE and norm(eps=-1.0) == SHAPE and norm(eps=INF) == SHAPE and norm(eps=1e-40) == SHAPE and norm(eps=float("nan")) == SHAPE
    assert norm(x=None) == NULL and norm(w=None) == NULL and norm(h=None) == NULL and norm(s=None) == NULL and norm(q=None) == NULL
    assert norm(q=None, s=None) == NULL                      # neither codes nor values
    for name in ("x", "r", "w", "q", "h", "y"):
        assert norm(**{name: ODD}) == ALIGN, name
    for name in ("s", "rstd", "nf"):
        assert norm(**{name: UNEVEN}) == ALIGN, name
    assert norm(rows=0, x=None, q=None, s=None) == OK and norm(cols=0, x=None, q=None, s=None) == OK


def test_norm_backward_refusals():
    def b(dy=F, dt=0, h=F, hdt=0, rstd=F, w=F, wdt=0, dres=F, rows=4, cols=256, dx=F, dw=F, ws=F, wsb=1 << 40):
        return lib().rms_norm_backward(dy, dt, h, hdt, rstd, w, wdt, dres, rows, cols, dx, dw, ws, wsb, None)
    need = lib().rms_norm_backward_workspace_bytes(4, 256)
    assert need > 0 and lib().rms_norm_backward_workspace_bytes(4, 260) == 0 and lib().rms_norm_backward_workspace_bytes(-1, 256) == 0
    assert b(dt=2) == ENUM and b(hdt=2) == ENUM and b(wdt=2) == ENUM
    assert b(rows=-1) == SHAPE and b(cols=12) == SHAPE and b(cols=1 << 15) == SHAPE
    assert b(dy=None) == NULL and b(h=None) == NULL and b(rstd=None) == NULL and b(w=None) == NULL and b(dx=None) == NULL
    assert b(ws=None) == WS and b(wsb=need - 1) == WS and b(ws=ODD) == ALIGN
    for name in ("dy", "h", "w", "dres", "dx"):
        assert b(**{name: ODD}) == ALIGN, name
    assert b(rstd=UNEVEN) == ALIGN and b(dw=UNEVEN) == ALIGN
    assert b(rows=0, dw=None, dy=None, dx=None) == OK and b(cols=0, dy=None) == OK


def gate(x=F, dt=0, rows=4, cols=256, act=0, fmt=0, flags=0, q=F, s=F, y=None, nf=None, dy=F, back=False):
    if back:
        return lib().gated_act_backward(dy, x, dt, rows, cols, act, fmt, flags, q, s, y, nf, None)
    return lib().gated_act_quantize(x, dt, rows, cols, act, fmt, flags, q, s, y, nf, None)


@pytest.mark.parametrize("back", [False, True])
def test_gate_refusals(back):
    def g(**k):
        return gate(back=back, **k)
    assert g(dt=2) == ENUM and g(act=2) == ENUM and g(fmt=5) == ENUM and g(flags=3) == ENUM
    assert g(rows=-1) == SHAPE and g(cols=-8) == SHAPE and g(cols=252) == SHAPE
    assert g(rows=1 << 28, cols=256) == SHAPE and g(rows=1 << 30, cols=256) == SHAPE and g(rows=1 << 31, cols=8) == SHAPE and g(rows=1, cols=1 << 30) == SHAPE
    assert g(x=None) == NULL and g(q=None) == NULL and g(s=None) == NULL and g(q=None, s=None) == NULL
    assert g(x=ODD) == ALIGN and g(q=ODD) == ALIGN and g(y=ODD) == ALIGN and g(s=UNEVEN) == ALIGN and g(nf=UNEVEN) == ALIGN
    assert g(rows=0, x=None, q=None, s=None) == OK and g(cols=0, x=None) == OK
    if back:
        assert g(dy=None) == NULL and g(dy=ODD) == ALIGN and g(cols=264) == SHAPE     # codes of halves with a partial group


def test_layer_refusals():
    def f(x=F, t=4, d=256, w1=F, s1=F, w2=F, s2=F, e=8, h=128, fmt=0, act=0, ids=F, w=F, k=2, y=F, ws=F, wsb=1 << 40):
        return lib().expert_layer_tokens(x, t, d, w1, s1, w2, s2, e, h, fmt, act, ids, w, k, y, ws, wsb, None)
    need = lib().expert_layer_tokens_workspace_bytes(4, 2, 8, 256, 128)
    assert need >= 4 * 2 * 128 * 2 and lib().expert_layer_tokens_workspace_bytes(65, 2, 8, 256, 128) == 0
    assert f(fmt=2) == ENUM and f(act=2) == ENUM
    assert f(t=-1) == SHAPE and f(t=65) == SHAPE and f(d=264) == SHAPE and f(d=32784) == SHAPE and f(h=136) == SHAPE
    assert f(h=32784) == SHAPE and f(e=0) == SHAPE and f(e=1025) == SHAPE and f(k=0) == SHAPE and f(k=65) == SHAPE
    assert f(t=64, k=17) == SHAPE and f(d=-16) == SHAPE and f(h=-16) == SHAPE
    for name in ("x", "w1", "s1", "w2", "s2", "ids", "w", "y"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: UNEVEN}) == ALIGN, name
    for name in ("x", "w1", "w2", "y", "ws"):
        assert f(**{name: ODD}) == ALIGN, name
    assert f(ws=None) == WS and f(wsb=need - 1) == WS
    assert f(t=0, x=None, ids=None, y=None, ws=None) == OK and f(d=0, x=None, ws=None) == OK


class Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def clip(*entries, max_norm=1.0, norm=F, nf=None, ws=F, wsb=1 << 40, count=None, null=False):
    a = (Grad * max(1, len(entries)))(*[Grad(*e) for e in entries])
    return lib().clip_grads(None if null else ctypes.byref(a), len(entries) if count is None else count, max_norm, norm, nf, ws, wsb, None)


def test_clip_refusals():
    good = (0x10000, 0x20000, 100, 0, 0)
    assert clip(good, (0x10000, 0x20000, 5, 2, 0)) == ENUM and clip((0x10000, 0x20000, 5, -1, 0)) == ENUM
    assert clip(good, max_norm=0.0) == SHAPE and clip(good, max_norm=-1.0) == SHAPE and clip(good, max_norm=float("nan")) == SHAPE
    assert clip((0x10000, 0x20000, -1, 0, 0)) == SHAPE and clip((0x10000, 0x20000, 1 << 36, 0, 0)) == SHAPE
    assert clip(good, count=-1) == SHAPE and clip(good, count=(1 << 20) + 1) == SHAPE
    assert clip((None, 0x20000, 5, 0, 0)) == NULL and clip(count=1, null=True) == NULL
    assert clip(good, (0x10000, None, 5, 0, 0)) == NULL                  # some written and some not
    assert clip((0x10001, 0x20000, 5, 0, 0)) == ALIGN and clip((0x10002, 0x20000, 5, 1, 0)) == ALIGN
    assert clip((0x10000, 0x20002, 5, 1, 0)) == ALIGN and clip(good, norm=UNEVEN) == ALIGN and clip(good, nf=UNEVEN) == ALIGN
    assert clip(good, ws=None) == WS and clip(good, wsb=16) == WS and clip(good, ws=ODD) == ALIGN
    assert clip((0x10000, None, 100, 0, 0), norm=None) == OK             # nothing asked for
    assert ctypes.sizeof(Grad) == 32


def test_python_refusals():
    """No CPU path, and shapes are checked before the library is called."""
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.ones(256)
    with pytest.raises(TypeError):
        qf8.rms_norm_quantize(bf, w, qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.rms_norm_quantize(bf.half(), w, qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.rms_norm_backward(bf, bf, torch.ones(4), w)
    with pytest.raises(TypeError):
        qf8.gated_act_quantize(bf, qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.gated_act_backward(bf, bf, qf8.E4M3)
    u8 = torch.zeros(2, 8, 8, dtype=torch.uint8)
    with pytest.raises(TypeError):
        qf8.expert_layer_tokens(bf, u8, w, u8, w, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.clip_grads([w], 1.0)
    with pytest.raises(TypeError):
        qf8.grad_norm([w.long()])
    with pytest.raises(ValueError):
        qf8.grad_norm([])
    with pytest.raises(ValueError):
        qf8.clip_grads([w], 1.0, out=[])
