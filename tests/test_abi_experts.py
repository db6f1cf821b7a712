"""Refusals of the products' and the expert layer's entry points (CPU: nothing is launched)."""
import ctypes

import pytest
import torch

import mx_block_scaled_amax_amd as qf8

OK, NULL, ENUM, SHAPE, ALIGN, WS = 0, -1, -2, -3, -4, -5
F = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
UNEVEN = ctypes.c_void_p(0x10002)


def lib():
    return qf8._load()


def mm(a=F, sa=F, b=F, sb=F, m=64, n=128, k=256, fa=0, fb=0, kind=0, flags=0, y=F, out=0, ws=None, wsb=0):
    return lib().matmul_block(a, sa, b, sb, m, n, k, fa, fb, kind, flags, y, out, ws, wsb, None)


def test_matmul_refusals():
    assert mm(fa=2) == ENUM and mm(fb=-1) == ENUM and mm(kind=3) == ENUM and mm(flags=2) == ENUM and mm(out=2) == ENUM
    assert mm(m=-1) == SHAPE and mm(k=6) == SHAPE and mm(n=-4) == SHAPE and mm(kind=1, n=126) == SHAPE
    assert mm(n=1 << 23) == SHAPE and mm(k=1 << 23) == SHAPE and mm(m=1 << 31) == SHAPE
    assert mm(y=None) == NULL and mm(a=None) == NULL and mm(sb=None) == NULL
    assert mm(m=0, a=None, y=None) == OK and mm(n=0, b=None, y=None) == OK
    big = dict(m=8, n=128, k=65536, kind=1)
    need = lib().matmul_block_workspace_bytes(8, 128, 65536, 1, 0)
    assert need > 0
    assert mm(**big) == WS and mm(ws=F, wsb=need - 1, **big) == WS and mm(ws=ODD, wsb=need, **big) == ALIGN
    args = dict(ws=F, wsb=1 << 40)
    assert mm(a=ODD, **args) == ALIGN and mm(b=ODD, **args) == ALIGN and mm(y=ODD, **args) == ALIGN
    assert mm(sa=UNEVEN, **args) == ALIGN
    assert lib().matmul_block_workspace_bytes(-1, 4, 4, 0, 0) == 0 and lib().matmul_block_workspace_bytes(0, 4, 4, 0, 1) == 0


def me(a=F, sa=F, tokens=64, b=F, sb=F, offsets=F, experts=8, rows=F, nrows=128, n=128, k=256, fa=0, fb=0, kind=0, flags=0,
       y=F, out=0):
    return lib().matmul_block_experts(a, sa, tokens, b, sb, offsets, experts, rows, nrows, n, k, fa, fb, kind, flags, y,
                                      out, None)


def test_matmul_experts_refusals():
    assert me(kind=2) == ENUM and me(fa=9) == ENUM and me(flags=4) == ENUM
    assert me(experts=0) == SHAPE and me(experts=1025) == SHAPE and me(rows=None, tokens=127) == SHAPE
    assert me(tokens=1 << 25, k=256) == SHAPE and me(k=2) == SHAPE and me(kind=1, n=6) == SHAPE and me(tokens=-1) == SHAPE
    assert me(offsets=None) == NULL and me(y=None) == NULL and me(a=None) == NULL and me(b=None) == NULL
    assert me(nrows=0, y=None) == OK
    assert me(a=ODD) == ALIGN and me(offsets=UNEVEN) == ALIGN and me(rows=UNEVEN) == ALIGN


def test_matmul_experts_wgrad_refusals():
    def wg(at=F, sat=F, bt=F, sbt=F, offsets=F, experts=4, nrows=256, m=64, n=64, fa=0, fb=0, flags=0, y=F, out=1):
        return lib().matmul_block_experts_wgrad(at, sat, bt, sbt, offsets, experts, nrows, m, n, fa, fb, flags, y, out, None)
    assert wg(fa=2) == ENUM and wg(out=3) == ENUM and wg(flags=8) == ENUM
    assert wg(nrows=130) == SHAPE and wg(experts=0) == SHAPE and wg(m=-1) == SHAPE
    assert wg(at=None) == NULL and wg(offsets=None) == NULL and wg(y=None) == NULL
    assert wg(bt=ODD) == ALIGN and wg(m=0, y=None) == OK


def test_route_refusals():
    def r(x=F, dt=0, t=4, e=64, k=8, score=0, bias=None, g=1, tg=1, ids=F, w=F):
        return lib().route_experts(x, dt, t, e, k, score, bias, g, tg, 1, 1.0, ids, w, None)
    assert r(dt=2) == ENUM and r(score=2) == ENUM
    assert r(t=-1) == SHAPE and r(e=0) == SHAPE and r(e=1025) == SHAPE and r(k=0) == SHAPE and r(k=65, e=128) == SHAPE
    assert r(g=3) == SHAPE and r(g=8, tg=9) == SHAPE and r(g=8, tg=0) == SHAPE
    assert r(k=8, e=8, g=4, tg=2) == SHAPE                       # 4 open experts, 8 asked for
    assert r(g=65, e=130) == SHAPE and r(k=9, e=8) == SHAPE
    assert r(x=None) == NULL and r(ids=None) == NULL and r(w=None) == NULL
    assert r(t=0, x=None) == OK and r(bias=UNEVEN) == ALIGN

    def b(x=F, dt=0, t=4, e=64, ids=F, dw=F, k=8, score=0, d=F):
        return lib().route_experts_backward(x, dt, t, e, ids, dw, k, score, 1, 1.0, d, None)
    assert b(dt=5) == ENUM and b(k=0) == SHAPE and b(k=65, e=64) == SHAPE and b(d=None) == NULL and b(ids=UNEVEN) == ALIGN


def test_order_refusals():
    def o(ids=F, t=4, k=2, e=8, align=16, off=F, rows=F, nrows=None, slots=F, ws=None, wsb=0):
        if nrows is None:
            nrows = lib().order_experts_rows(t, k, e, align)
        return lib().order_experts(ids, t, k, e, align, off, rows, nrows, slots, ws, wsb, None)
    assert lib().order_experts_rows(4, 2, 8, 16) == 128 and lib().order_experts_rows(0, 2, 8, 16) == 0
    assert lib().order_experts_rows(10, 2, 8, 1) == 20 and lib().order_experts_rows(10, 2, 2000, 1) == 0
    assert o(align=0) == SHAPE and o(align=1025) == SHAPE and o(e=0) == SHAPE and o(e=1025) == SHAPE and o(k=0) == SHAPE
    assert o(nrows=127) == SHAPE and o(t=1 << 30, k=8) == SHAPE
    assert o(ids=None) == NULL and o(off=None) == NULL and o(rows=None) == NULL and o(slots=None) == NULL
    need = lib().order_experts_workspace_bytes(4096, 8, 64)
    assert need > 0 and o(t=4096, k=8, e=64) == WS and o(t=4096, k=8, e=64, ws=F, wsb=need - 1) == WS
    assert o(t=4096, k=8, e=64, ws=ODD, wsb=need) == ALIGN and o(slots=UNEVEN) == ALIGN


def test_combine_refusals():
    def c(x=F, dt=0, r=64, d=128, w=F, s=F, t=8, k=4, y=F):
        return lib().combine_experts(x, dt, r, d, w, s, t, k, y, None)
    assert c(dt=2) == ENUM and c(r=-1) == SHAPE and c(d=-1) == SHAPE and c(k=0) == SHAPE and c(k=65) == SHAPE
    assert c(x=None) == NULL and c(w=None) == NULL and c(s=None) == NULL and c(y=None) == NULL
    assert c(t=0, y=None) == OK and c(d=0, y=None) == OK and c(x=ODD) == ALIGN and c(y=ODD) == ALIGN

    def b(dy=F, x=F, dt=0, r=64, d=128, w=F, s=F, rows=F, t=8, k=4, dx=F, dw=F):
        return lib().combine_experts_backward(dy, x, dt, r, d, w, s, rows, t, k, dx, dw, None)
    assert b(dt=2) == ENUM and b(k=0) == SHAPE and b(rows=None) == NULL and b(dy=None) == NULL and b(dw=None) == NULL
    assert b(dx=ODD) == ALIGN and b(dw=UNEVEN) == ALIGN and b(t=0, r=0, dy=None, dw=None) == OK


def test_python_refusals():
    """No CPU path, and shapes are checked before the library is called."""
    u8, f32, i32 = (lambda *s: torch.zeros(*s, dtype=torch.uint8)), torch.zeros, (lambda *s: torch.zeros(*s, dtype=torch.int32))
    with pytest.raises(TypeError):
        qf8.matmul_block(u8(4, 128), f32(4, 1), u8(8, 128), f32(1, 1), qf8.E4M3, qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.matmul_block_experts(u8(4, 128), f32(4, 1), u8(2, 8, 128), f32(2, 1, 1), i32(3), qf8.E4M3, qf8.E4M3)
    with pytest.raises(TypeError):
        qf8.route_experts(f32(4, 8), 2)
    with pytest.raises(TypeError):
        qf8.order_experts(i32(4, 2), 8)
    with pytest.raises(TypeError):
        qf8.combine_experts(f32(4, 8), f32(2, 2), i32(2, 2))
