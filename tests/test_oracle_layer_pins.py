"""Pins for the fp64 oracle of the operators around the attention (``oracle/layer.py``): closed
forms, finite differences of every gradient, and identities that do not use the oracle's own
steps."""
import numpy as np
import pytest

from oracle import layer as L


def r(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape)


def gates(seed, *shape):
    return np.random.default_rng(seed).uniform(0.2, 1.0, size=shape)


def differences(f, x, grad, seed, eps=1e-6):
    """The gradient against central differences along random directions."""
    for k in range(4):
        d = r(seed + k, *x.shape)
        num = (f(x + eps * d) - f(x - eps * d)) / (2 * eps)
        assert num == pytest.approx(float((grad * d).sum()), rel=1e-6, abs=1e-7)


def test_constant_gate_is_the_geometric_sum():
    x, a = r(1, 2, 9, 3), 0.7
    h, last, _ = L.linear_scan(x, np.full_like(x, a))
    want = sum(a ** (8 - s) * x[:, s] for s in range(9))
    np.testing.assert_allclose(last, want, rtol=1e-13)
    np.testing.assert_allclose(L.linear_scan(x, np.ones_like(x))[0], x.cumsum(1), rtol=1e-12)
    # the blend with constant input tends to the input
    h, _, _ = L.linear_scan(np.full((1, 400, 1), 3.0), np.full((1, 400, 1), a), blend=True)
    assert h[0, -1, 0] == pytest.approx(3.0)


@pytest.mark.parametrize("blend", [False, True])
def test_split_and_packed_continue(blend):
    x, a, h0 = r(2, 2, 13, 4), gates(3, 2, 13, 4), r(4, 2, 4)
    h, last, _ = L.linear_scan(x, a, h0, blend)
    u, mid, _ = L.linear_scan(x[:, :5], a[:, :5], h0, blend)
    v, end, _ = L.linear_scan(x[:, 5:], a[:, 5:], mid, blend)
    np.testing.assert_array_equal(np.concatenate([u, v], 1), h)
    p, ends, _ = L.linear_scan_packed(x.reshape(26, 4), a.reshape(26, 4), [0, 13, 13, 26], np.stack([h0[0], h0[1], h0[1]]),
                                      blend)
    np.testing.assert_array_equal(p.reshape(2, 13, 4), h)
    np.testing.assert_array_equal(ends[[0, 2]], last)
    np.testing.assert_array_equal(ends[1], h0[1])


@pytest.mark.parametrize("blend", [False, True])
def test_scan_gradients_by_differences(blend):
    x, a, h0, dh, ds = r(5, 2, 7, 3), gates(6, 2, 7, 3), r(7, 2, 3), r(8, 2, 7, 3), r(9, 2, 3)

    def loss(x, a, h0):
        h, last, _ = L.linear_scan(x, a, h0, blend)
        return float((h * dh).sum() + (last * ds).sum())

    (dx, da, d0), _ = L.linear_scan_backward(x, a, dh, h0, ds, blend)
    differences(lambda v: loss(v, a, h0), x, dx, 10)
    differences(lambda v: loss(x, v, h0), a, da, 20)
    differences(lambda v: loss(x, a, v), h0, d0, 30)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_identities(interleaved):
    x, pos, f = r(11, 2, 3, 5, 10), np.random.default_rng(12).integers(0, 900, size=(2, 5)), np.array([1.0, 0.1, 0.01])
    y, _ = L.rotary(x, pos, f, 1.3, interleaved)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    np.testing.assert_allclose((y[..., :6] ** 2).sum(-1), 1.69 * (x[..., :6] ** 2).sum(-1), rtol=1e-12)
    back, _ = L.rotary(y, pos, f, 1 / 1.3, interleaved, transpose=True)
    np.testing.assert_allclose(back, x, atol=1e-12)
    # products of q and k depend on the distance of their positions alone
    q, k = r(13, 1, 1, 1, 6), r(14, 1, 1, 1, 6)
    dot = [float((L.rotary(q, [[p + 7]], f, 1, interleaved)[0] * L.rotary(k, [[p]], f, 1, interleaved)[0]).sum())
           for p in (0, 3, 500)]
    np.testing.assert_allclose(dot, dot[0], rtol=1e-10)
    # the two pair layouts are one operator on permuted values
    perm = [0, 2, 4, 1, 3, 5, 6, 7, 8, 9] if interleaved else [0, 3, 1, 4, 2, 5, 6, 7, 8, 9]
    other, _ = L.rotary(x[..., perm], pos, f, 1.3, not interleaved)
    np.testing.assert_allclose(other, y[..., perm], rtol=1e-13)


def test_norm_closed_forms_and_gradients():
    w = 1 + 0.3 * r(15, 8)
    y, _ = L.rms_norm(np.full((1, 8), -5.0), np.ones(8), eps=0.0)
    np.testing.assert_allclose(y, -1.0)
    h, dy, dres = r(16, 2, 3, 8), r(17, 2, 3, 8), r(18, 2, 3, 8)
    np.testing.assert_allclose((L.rms_norm(h, np.ones(8), 0.0)[0] ** 2).mean(-1), 1.0)
    (dx, dw), _ = L.rms_norm_backward(h, w, dy, dres, 1e-3)
    differences(lambda v: float((L.rms_norm(v, w, 1e-3)[0] * dy).sum() + (v * dres).sum()), h, dx, 40)
    differences(lambda v: float((L.rms_norm(h, v, 1e-3)[0] * dy).sum()), w, dw, 50)
