"""GPU parity of the RMS norm with residual and 8-bit output (``la_rms_norm*``) against the fp64
oracle.

Tolerance, element by element: the oracle's bound plus half a step of the output's type.  e4m3
values: half a step is 2^-4 of the value, or 2^-10 (half the smallest subnormal); a scale is off
by the bound of its largest y.
"""
import numpy as np
import pytest
import torch

from oracle import layer as L
from parity_util import f64

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def la():
    import gated_delta_rule_attention_b200 as m
    m.library()
    return m


def close(y, ref, bound):
    half = HALF[y.dtype]
    y = f64(y)
    bad = ~(np.abs(y - ref) <= bound * (1 + half) + half * np.abs(ref))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst error {np.abs(y - ref).max():.3e}"


def close_fp8(q, scales, ref, bound, group):
    """q e4m3 [.., C], scales [.., C / group] against y [.., C]."""
    parts = ref.reshape(*scales.shape, group)
    top = np.abs(parts).max(-1)
    want = np.where(top > 0, np.maximum(top / 448, 2.0 ** -126), 1.0)
    s = f64(scales)
    assert (np.abs(s - want) <= 100 * L.EPS * want).all()
    exact = parts / want[..., None]
    got = f64(q.float()).reshape(parts.shape)
    assert np.isfinite(got).all() and np.abs(got).max(initial=0) <= 448
    slack = bound.reshape(parts.shape) / want[..., None] + 100 * L.EPS * np.abs(exact)
    bad = ~(np.abs(got - exact) <= np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** -10) + slack * (1 + 2.0 ** -4))
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside"


def rand(dtype, *shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# every width of a row: parts of a warp, a warp, a CTA; odd columns; rows that fill no block
SIZES = [(1, 1), (3, 7), (1, 8), (5, 64), (40, 72), (33, 128), (2, 200), (100, 256), (9, 300), (7, 512), (4, 520),
         (3, 1024), (5, 1000), (2, 1001), (3, 2048), (4, 2056), (2, 2050), (3, 4096), (2, 5000), (1, 4097),
         (2, 8192), (1, 8200), (1, 16384), (1, 16383), (700, 136)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", SIZES)
def test_norm_matches_oracle(la, dtype, R, C):
    x, res, w = rand(dtype, R, C, seed=C), 3 * rand(dtype, R, C, seed=C + 1), 1 + 0.3 * rand(torch.float32, C, seed=2)
    y = la.rms_norm(x, w)
    z, h = la.rms_norm(x, w, residual=res, eps=1e-3)
    q, s = la.rms_norm(x, w, fp8=True)
    qr, sr, hr = la.rms_norm(x, w, residual=res, fp8=True, eps=1e-3)
    la.check_status()
    close(y, *L.rms_norm(f64(x), f64(w)))
    assert torch.equal(h, (x.float() + res.float()).to(dtype)) and torch.equal(h, hr)
    close(z, *L.rms_norm(f64(h), f64(w), 1e-3))
    assert q.dtype == torch.float8_e4m3fn and s.shape == (R, 1)
    close_fp8(q, s, *L.rms_norm(f64(x), f64(w)), C)
    close_fp8(qr, sr, *L.rms_norm(f64(h), f64(w), 1e-3), C)
    if C % 128 == 0:
        q, s = la.rms_norm(x, w, fp8=True, group=128)
        qr, sr, _ = la.rms_norm(x, w, residual=res, fp8=True, group=128, eps=1e-3)
        la.check_status()
        assert s.shape == (R, C // 128)
        close_fp8(q, s, *L.rms_norm(f64(x), f64(w)), 128)
        close_fp8(qr, sr, *L.rms_norm(f64(h), f64(w), 1e-3), 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", SIZES + [(3000, 256), (5000, 8), (1300, 1000), (700, 2048)])
def test_norm_backward_matches_oracle(la, dtype, R, C):
    h, dy, dres = (rand(dtype, R, C, seed=C + i) for i in range(3))
    w = 1 + 0.3 * rand(torch.float32, C, seed=2)
    for extra in (None, dres):
        dx, dw = la.rms_norm_backward(h, w, dy, dresidual=extra, eps=1e-4)
        la.check_status()
        refs, bounds = L.rms_norm_backward(f64(h), f64(w), f64(dy), None if extra is None else f64(extra), 1e-4)
        close(dx, refs[0], bounds[0])
        close(dw, refs[1], bounds[1])
        again = la.rms_norm_backward(h, w, dy, dresidual=extra, eps=1e-4)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 128), (2, 3, 5, 64), (1, 16, 33, 128), (3, 2, 50, 128), (2, 5, 7, 24),
                                   (1, 4, 9, 10), (2, 2, 3, 256)])
def test_norm_heads_matches_oracle(la, dtype, shape):
    B, H, T, d = shape
    x, w = rand(dtype, *shape, seed=T), 1 + 0.3 * rand(torch.float32, d, seed=1)
    y = la.rms_norm_heads(x, w)
    q, s = la.rms_norm_heads(x, w, fp8=True)
    dy = rand(dtype, B, T, H * d, seed=3)
    dx, dw = la.rms_norm_heads_backward(x, w, dy)
    la.check_status()
    ref, b = (np.moveaxis(v, 1, 2) for v in L.rms_norm(f64(x), f64(w)))
    close(y, ref.reshape(B, T, -1), b.reshape(B, T, -1))
    assert s.shape == (B, T, H)
    close_fp8(q, s, ref, b, d)
    refs, bounds = L.rms_norm_backward(f64(x), f64(w), np.moveaxis(f64(dy).reshape(B, T, H, d), 2, 1))
    close(dx, refs[0], bounds[0])
    close(dw, refs[1], bounds[1])


def test_norm_residual_in_place(la):
    x, res, w = rand(torch.bfloat16, 50, 2048, seed=1), rand(torch.bfloat16, 50, 2048, seed=2), torch.ones(2048, device="cuda")
    y, h = la.rms_norm(x, w, residual=res)
    r2 = res.clone()
    y2, h2 = la.rms_norm(x, w, residual=r2, residual_out=r2)
    x3 = x.clone()
    y3, h3 = la.rms_norm(x3, w, residual=res, residual_out=x3)
    la.check_status()
    assert h2.data_ptr() == r2.data_ptr() and h3.data_ptr() == x3.data_ptr()
    for a, b in ((y2, h2), (y3, h3)):
        assert torch.equal(a, y) and torch.equal(b, h)


@pytest.mark.parametrize("C", [128, 2048, 9])
def test_norm_zero_tiny_and_huge_rows(la, C):
    """Zero rows (eps alone holds the root), rows at the bottom and the top of bf16's range, and a
    row with an infinity and one with a NaN, which stay in their rows."""
    w = torch.ones(C, device="cuda")
    x = rand(torch.bfloat16, 8, C, seed=4)
    clean = la.rms_norm(x, w)
    x[0] = 0
    x[1] = 1e-38
    x[2] = 1e15
    x[3, 1] = float("inf")
    x[4, 2] = float("nan")
    y = la.rms_norm(x, w)
    q, s = la.rms_norm(x, w, fp8=True)
    la.check_status()
    assert (y[0] == 0).all() and (q[0].float() == 0).all() and (s[0] == 1).all()
    assert (y[1].float() - 1e-35).abs().max() < 1e-37 and torch.isfinite(q[1].float()).all()
    assert (y[2] == 1).all() and (q[2].float() == 448).all()
    assert torch.isnan(y[3, 1]) and torch.isnan(y[4]).all()
    assert torch.isnan(q[3, 1].float()) and torch.isnan(q[4].float()).all()
    assert torch.equal(y[5:], clean[5:])
    # gradients of a zero row: eps alone scales them
    dx, dw = la.rms_norm_backward(x[:1], w, torch.ones_like(x[:1]), eps=1e-4)
    la.check_status()
    assert (dx == 100).all() and (dw == 0).all()


def test_norm_empty_and_refusals(la):
    w = torch.ones(64, device="cuda")
    assert la.rms_norm(torch.zeros(0, 64, device="cuda"), w).shape == (0, 64)
    dx, dw = la.rms_norm_backward(torch.zeros(0, 64, device="cuda"), w, torch.zeros(0, 64, device="cuda"))
    la.check_status()
    assert dx.shape == (0, 64) and (dw == 0).all()
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(la.LaError, match="UNSUPPORTED"):
        la.rms_norm(torch.zeros(1, 16392, device="cuda"), torch.ones(16392, device="cuda"))
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.rms_norm(torch.zeros(257, device="cuda")[1:].view(4, 64), w)
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.rms_norm(x, w, residual=x.clone(), residual_out=torch.zeros(4, 64))
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.rms_norm(x, w, eps=-1.0)
    lib, p = la.library(), (lambda t: t.data_ptr())
    assert lib.la_rms_norm(0, 1, 1, 4, 64, p(x), None, p(w), 1e-6, None, p(x), None, 0, 0, None) == 1   # y on x
    assert lib.la_rms_norm_backward(0, 1, 1, 4, 64, p(x), p(w), 1e-6, p(x), None, p(torch.zeros_like(x)), p(w), p(w), 256, None) == 1
    la.check_status()


def test_norm_gradient_against_differences(la):
    """The backward kernel against differences of the forward kernel in fp32 (a step of 2^-6 along
    a direction: truncation of the second order)."""
    x, w, dy = rand(torch.float32, 6, 40, seed=1), 1 + 0.3 * rand(torch.float32, 40, seed=2), rand(torch.float32, 6, 40, seed=3)
    dx, dw = la.rms_norm_backward(x, w, dy)
    e = 2.0 ** -6
    for t, grad, f in ((x, dx, lambda v: la.rms_norm(v, w)), (w, dw, lambda v: la.rms_norm(x, v))):
        d = rand(torch.float32, *t.shape, seed=5)
        num = float(((f(t + e * d).double() - f(t - e * d).double()) * dy).sum()) / (2 * e)
        want = float((grad.double() * d).sum())
        assert num == pytest.approx(want, rel=2e-3, abs=2e-3 * float((grad.double() * d).norm()))


def test_norm_offsets_beyond_32_bits(la):
    R, C = 2 ** 31 // 1024 + 9, 1024
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    w = 1 + 0.3 * rand(torch.float32, C, seed=2)
    y, h = la.rms_norm(x, w, residual=x)
    tail = la.rms_norm(x[-20:], w, residual=x[-20:])
    assert torch.equal(y[-20:], tail[0]) and torch.equal(h[-20:], tail[1])
    q, s = la.rms_norm(x, w, fp8=True, group=128)
    qt, st = la.rms_norm(x[-20:], w, fp8=True, group=128)
    assert torch.equal(q[-20:].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s[-20:], st)
    dx, _ = la.rms_norm_backward(x, w, h)
    assert torch.equal(dx[-20:], la.rms_norm_backward(x[-20:], w, h[-20:])[0])
    T = 2 ** 31 // 256 + 5   # two heads of 128
    o = x.view(-1)[:2 * T * 128].view(1, 2, T, 128)
    yh = la.rms_norm_heads(o, w[:128].contiguous())
    for head in (0, 1):
        want = la.rms_norm(o[0, head, -9:], w[:128].contiguous())
        assert torch.equal(yh[0, -9:, head * 128:(head + 1) * 128], want)
    la.check_status()
