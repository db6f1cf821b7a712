"""The norm of a residual stream against its definition in 64 bits.

Tolerances. An fp32 sum of squares of at most 16384 terms, 64 to a thread and 22 joins, is within 2^-17 of the exact one;
R within half of that and four roundings, y within two more: rel(y) <= 2^-17. A scale is off by that and its own 2^-24, a
code by its half step (E4M3 2^-4 and at least 2^-10, E5M2 2^-3 and 2^-17) at a value off by 2^-16 of itself. With FP32 x the values
y are there too, and the codes are quantize_block's of them bit for bit. dx: its type's half step, and 2^-17 of the sum of its terms'
magnitudes; dweight: (rows + 16) 2^-24 of the sum of the terms' magnitudes, in any order of summation."""
import pytest
import torch

import mx_block_scaled_amax_amd as qf8

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
F8 = {qf8.E4M3: (torch.float8_e4m3fn, 448.0, 2.0 ** -4, 2.0 ** -10), qf8.E5M2: (torch.float8_e5m2, 57344.0, 2.0 ** -3, 2.0 ** -17)}


def made(rows, cols, x=BF, residual=None, w=BF, seed=0, spread=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    a = (normal(rows, cols) * torch.exp(spread * normal(rows, 1))).to(x)
    r = None if residual is None else (2 * normal(rows, cols)).to(residual)
    return a, (1 + 0.3 * normal(cols)).to(w), r, normal


def exact(x, w, r, eps):
    h = x.double() if r is None else (x.float() + r.float()).to(r.dtype).double()
    rstd = 1 / (h.square().mean(1) + eps).sqrt()
    return h, rstd, h * rstd[:, None] * w.double()


def check_codes(q, scales, y, fmt, pow2):
    dt, top, half, least = F8[fmt]
    rows, cols = y.shape
    pad = torch.nn.functional.pad(y, (0, -cols % 128)).view(rows, -1, 128)
    amax = pad.abs().amax(2)
    s = torch.where(amax > 0, top / amax, 1.0)
    if pow2:                                               # off by 2 only next to a border
        low = torch.exp2(torch.floor(torch.log2(s * (1 - 2.0 ** -16))))
        high = torch.exp2(torch.floor(torch.log2(s * (1 + 2.0 ** -16))))
        assert bool(((scales == torch.where(amax > 0, low, 1.0)) | (scales == torch.where(amax > 0, high, 1.0))).all())
    else:
        assert bool(((scales - s).abs() <= 2.0 ** -16 * s).all())
    v = y * scales.double().repeat_interleave(128, 1)[:, :cols]
    got = q.view(dt).double()
    assert bool(((got - v).abs() <= torch.clamp(half * v.abs(), min=least) * (1 + 2.0 ** -9) + 2.0 ** -16 * v.abs()).all())


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 7168), (3, 128), (5, 136), (130, 512), (9, 520), (33, 1024), (2, 1032),
                                       (4, 2048), (7, 2056), (301, 4096), (5, 4104), (3, 8192), (2, 8200), (3, 16384), (2050, 16)])
@pytest.mark.parametrize("x,residual,w", [(BF, None, BF), (BF, BF, F32), (BF, F32, BF), (F32, BF, F32), (F32, None, F32), (F32, F32, BF)])
def test_forward(rows, cols, x, residual, w):
    a, wt, r, _ = made(rows, cols, x, residual, w, seed=rows + cols)
    keep = None if r is None else r.clone()
    fmt = qf8.E5M2 if cols % 16 else qf8.E4M3
    pow2 = rows % 2 == 0
    got = qf8.rms_norm_quantize(a, wt, fmt, residual=r, eps=1e-5, pow2_scales=pow2, want_y=True, want_rstd=True)
    h, rstd, y = exact(a, wt, r, 1e-5)
    if r is None:
        assert got.h is a
    else:
        assert torch.equal(got.h.double(), h) and torch.equal(r, keep)
    assert bool(((got.rstd.double() - rstd).abs() <= 2.0 ** -17 * rstd).all())
    assert bool(((got.y.double() - y).abs() <= (HALF[x] * (1 + 2.0 ** -16) + 2.0 ** -17) * y.abs()).all())
    check_codes(got.q, got.scales, y, fmt, pow2)
    if x == F32:
        q, s, _ = qf8.quantize_block(got.y, 1, 128, fmt, want_amax=False, pow2_scales=pow2)
        assert torch.equal(q, got.q) and torch.equal(s, got.scales)


@pytest.mark.parametrize("cols", [1032, 4096, 4104, 7168, 8192, 8200, 16384])
def test_a_row_by_itself(cols):
    """A row's bits do not hang on how many rows there are."""
    a, w, r, _ = made(700, cols, BF, F32, F32, seed=cols)
    every = qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=r, want_rstd=True)
    for rows in (slice(0, 1), slice(300, 500), slice(699, 700)):
        some = qf8.rms_norm_quantize(a[rows].contiguous(), w, qf8.E4M3, residual=r[rows].contiguous(), want_rstd=True)
        assert torch.equal(some.rstd, every.rstd[rows]) and torch.equal(some.q, every.q[rows]) and torch.equal(some.scales, every.scales[rows])
    x = (a.float() * 2.0 ** 64).contiguous()                # squares beyond fp32
    big = qf8.rms_norm_quantize(x, w, None, want_rstd=True).rstd
    assert torch.equal(big[:3], qf8.rms_norm_quantize(x[:3].contiguous(), w, None, want_rstd=True).rstd)


def test_alone_and_in_place():
    a, w, r, _ = made(37, 1544, BF, BF, BF, seed=4)
    every = qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=r, want_y=True, want_rstd=True)
    only = qf8.rms_norm_quantize(a, w, None, residual=r)
    assert only.q is None and only.scales is None and only.rstd is None and torch.equal(only.y, every.y)
    codes = qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=r)
    assert codes.y is None and torch.equal(codes.q, every.q) and torch.equal(codes.scales, every.scales)
    stream = r.clone()
    place = qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=stream, h=stream)
    assert place.h is stream and torch.equal(stream, every.h) and torch.equal(place.q, every.q)


@pytest.mark.parametrize("cols", [264, 4096, 16384])
def test_ends_of_the_range(cols):
    """Zeros, squares beyond fp32, tiny rows, Inf and NaN: each row by itself."""
    x = torch.randn(8, cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x[1] = 0
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** -100
    x[4] = torch.finfo(F32).max
    x[5, 7] = float("inf")
    x[6, 3] = float("nan")
    x[7] = 0
    x[7, 0] = 1e30
    w = torch.full((cols,), 0.5, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qf8.rms_norm_quantize(x, w, qf8.E4M3, want_y=True, want_rstd=True, nonfinite=flag)
    fine = [0, 1, 2, 3, 4, 7]
    _, rstd, y = exact(x[fine], w, None, 1e-6)
    assert bool(((got.rstd[fine].double() - rstd).abs() <= 2.0 ** -17 * rstd).all())
    assert bool(((got.y[fine].double() - y).abs() <= 2.0 ** -16 * y.abs() + 2.0 ** -149).all())
    check_codes(got.q[fine], got.scales[fine], y, qf8.E4M3, False)
    assert flag.item() == 1 and bool((got.q[1] == 0).all()) and bool((got.scales[1] == 1).all())
    assert got.rstd[5].item() == 0 and bool(got.rstd[6].isnan())
    flag.zero_()
    qf8.rms_norm_quantize(x[fine], w, qf8.E4M3, nonfinite=flag)
    assert flag.item() == 0


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 4096), (3, 136), (4100, 128), (2101, 1000), (1030, 1032), (17, 2048), (1500, 4096),
                                       (5, 7168), (2, 8200), (1029, 16384)])
@pytest.mark.parametrize("dy,h,w,dres", [(BF, BF, BF, True), (BF, F32, F32, False), (F32, BF, F32, False), (F32, F32, BF, True)])
def test_backward(rows, cols, dy, h, w, dres):
    a, wt, _, normal = made(rows, cols, h, None, w, seed=rows * 3 + cols)
    g = (normal(rows, cols) * 1e-2).to(dy)
    res = (normal(rows, cols) * 1e-2).to(h) if dres else None
    rstd = (1 / (a.double().square().mean(1) + 1e-6).sqrt()).float()
    dx, dw = qf8.rms_norm_backward(g, a, rstd, wt, dres=res)
    r, n, gw = rstd.double()[:, None], a.double() * rstd.double()[:, None], g.double() * wt.double()
    mean = (gw * n).mean(1, keepdim=True)
    want = r * (gw - n * mean) + (0 if res is None else res.double())
    size = r * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True)) + (0 if res is None else res.double().abs())
    assert bool(((dx.double() - want).abs() <= HALF[h] * want.abs() + 2.0 ** -17 * size).all())
    terms = g.double() * n
    assert bool(((dw.double() - terms.sum(0)).abs() <= (rows + 16) * 2.0 ** -24 * terms.abs().sum(0)).all())
    assert torch.equal(dw, qf8.rms_norm_backward(g, a, rstd, wt, dres=res)[1])
    only, none = qf8.rms_norm_backward(g, a, rstd, wt, dres=res, want_dweight=False)
    assert none is None and torch.equal(only, dx)
    if res is not None:
        qf8.rms_norm_backward(g, a, rstd, wt, dres=res, dx=res)
        assert torch.equal(res, dx)


def test_gradients_against_differences():
    """The slope of <dy, y> along a direction: central differences of the definition in 64 bits, with a step of 2^-20
    (error 2^-40 times third derivatives), against the kernel's FP32 gradients (2^-16 of the terms)."""
    a, w, _, normal = made(6, 520, F32, None, F32, seed=9, spread=0.3)
    dy, along, wlong = normal(6, 520), normal(6, 520), normal(520)
    rstd = qf8.rms_norm_quantize(a, w, None, want_rstd=True).rstd
    dx, dw = qf8.rms_norm_backward(dy, a, rstd, w)

    def value(t):
        x, v = a.double() + t * along.double(), w.double() + t * wlong.double()
        return float((dy.double() * x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * v).sum())
    t = 2.0 ** -20
    slope = (value(t) - value(-t)) / (2 * t)
    terms = torch.cat([(dx.double() * along.double()).flatten(), dw.double() * wlong.double()])
    assert abs(float(terms.sum()) - slope) <= 2.0 ** -16 * float(terms.abs().sum())


def test_sizes_of_nothing():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    got = qf8.rms_norm_quantize(e, w, qf8.E4M3, residual=e, want_y=True, want_rstd=True)
    assert got.q.shape == (0, 64) and got.scales.shape == (0, 1) and got.rstd.shape == (0,)
    dx, dw = qf8.rms_norm_backward(e, e, torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(w))
    n = qf8.rms_norm_quantize(torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda"), qf8.E4M3)
    assert n.q.shape == (3, 0)


def test_refusals():
    a, w, r, _ = made(4, 264, BF, BF, BF)
    with pytest.raises(ValueError):
        qf8.rms_norm_quantize(a.t(), w, qf8.E4M3)
    with pytest.raises(ValueError):
        qf8.rms_norm_quantize(a, w[:256], qf8.E4M3)
    with pytest.raises(ValueError):
        qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=r[:3])
    with pytest.raises(ValueError):
        qf8.rms_norm_quantize(a, w, qf8.E4M3, h=r)
    with pytest.raises(TypeError):
        qf8.rms_norm_quantize(a, w, qf8.E4M3, residual=r, h=torch.empty_like(r, dtype=F32))
    with pytest.raises(qf8.QF8Error):
        qf8.rms_norm_quantize(a[:, :260].contiguous(), w[:260].contiguous(), qf8.E4M3)
    with pytest.raises(qf8.QF8Error):
        qf8.rms_norm_quantize(a, w, qf8.E4M3, eps=0.0)
    with pytest.raises(qf8.QF8Error):
        qf8.rms_norm_backward(a, a, torch.ones(4, device="cuda"), w, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
