"""fp64 oracle of the operators around the attention -- TEST INFRASTRUCTURE ONLY.

The gated linear recurrence with a vector state and its gradients, rotary positions, and the
root-mean-square norm with its gradients, each written out from its definition.  Every function
that a kernel is checked by also gives the bound of what fp32 arithmetic may add to the result:
``EPS`` (half an fp32 step) times the sum of the absolute values of everything that is added up,
each counted as often as a rounding can meet it.
"""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24


def _f64(x):
    return np.ascontiguousarray(np.asarray(x, dtype=np.float64))


def linear_scan(x, a, h0=None, blend=False):
    """h_t = a_t h_{t-1} + u_t over axis 1 of [B, T, C]: (h, h_T, bound).

    bound: a term u_s that reaches row t has passed t - s steps of one rounding each, or the
    products of gates and joins of segments that stand for them: at most two a row (a product and
    a sum), and 64 for the joins of threads (5), warps (8), cluster ranks (16), each two, and its
    own making.  With m_t = sum |u_s| prod a, n_t = sum (t - s) |u_s| prod a: 2 n_t + 64 m_t."""
    x, a = _f64(x), _f64(a)
    B, T, C = x.shape
    u = (1.0 - a) * x if blend else x
    h = np.zeros((B, C)) if h0 is None else _f64(h0).copy()
    m, n = np.abs(h), np.zeros((B, C))
    out, bound = np.empty_like(x), np.empty_like(x)
    for t in range(T):
        h = a[:, t] * h + u[:, t]
        n = a[:, t] * (n + m)
        m = a[:, t] * m + np.abs(u[:, t])
        out[:, t], bound[:, t] = h, EPS * (2 * n + 64 * m)
    return out, h, bound


def linear_scan_packed(x, a, cu, state=None, blend=False):
    """Each packed sequence by itself: (h, final states, bound); rows of no sequence are zero."""
    x, a = _f64(x), _f64(a)
    N = len(cu) - 1
    h, bound = np.zeros_like(x), np.zeros_like(x)
    last = np.zeros((N, x.shape[1])) if state is None else _f64(state).copy()
    for s in range(N):
        lo, hi = cu[s], cu[s + 1]
        if hi > lo:
            o, end, b = linear_scan(x[None, lo:hi], a[None, lo:hi], last[s][None], blend)
            h[lo:hi], bound[lo:hi], last[s] = o[0], b[0], end[0]
    return h, last, bound


def linear_scan_backward(x, a, dh, h0=None, dstate=None, blend=False):
    """(dx, da, dh0) and their bounds, by the reverse recurrence l_t = dh_t + a_{t+1} l_{t+1}."""
    x, a, dh = _f64(x), _f64(a), _f64(dh)
    B, T, C = x.shape
    h, _, hb = linear_scan(x, a, h0, blend)
    first = np.zeros((B, 1, C)) if h0 is None else _f64(h0)[:, None]
    prev = np.concatenate([first, h[:, :-1]], 1)
    prev_b = np.concatenate([np.zeros((B, 1, C)), hb[:, :-1]], 1)
    m = np.zeros((B, C)) if dstate is None else _f64(dstate).copy()
    mag, n = np.abs(m), np.zeros((B, C))
    lam, lam_b = np.empty_like(x), np.empty_like(x)
    for t in range(T - 1, -1, -1):
        lam[:, t] = dh[:, t] + m
        mag, n = np.abs(dh[:, t]) + mag, n + mag
        lam_b[:, t] = EPS * (2 * n + 64 * mag)
        m = a[:, t] * lam[:, t]
        mag, n = a[:, t] * mag, a[:, t] * n
    d = prev - x if blend else prev
    scale = 1.0 - a if blend else np.ones_like(a)
    dx, da = scale * lam, lam * d
    size = np.abs(prev) + (np.abs(x) if blend else 0.0)
    return ((dx, da, m), (np.abs(scale) * lam_b + 4 * EPS * np.abs(lam),
                          np.abs(d) * lam_b + np.abs(lam) * prev_b + 4 * EPS * np.abs(lam) * size,
                          a[:, 0] * lam_b[:, 0] + 4 * EPS * np.abs(m)))


def rotary(x, pos, freqs, scale=1.0, interleaved=False, transpose=False):
    """x [B, H, T, d] at positions [B, T]: (y, bound).  The angle in turns is at most 1/2, so its
    fp32 rounding moves sin and cos by at most 2 pi 2^-26 < 2 EPS; their own error, the products
    with the scale and of the pair, and the sum make at most 8 EPS of |u| + |v|."""
    x = _f64(x)
    r = 2 * len(freqs)
    ang = (np.asarray(pos, dtype=np.float64)[:, None, :, None] * _f64(freqs))
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if transpose else 1.0)
    y, bound = x.copy(), np.zeros_like(x)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, v = x[..., i], x[..., j]
    y[..., i], y[..., j] = scale * (u * c - v * s), scale * (u * s + v * c)
    b = 8 * EPS * abs(scale) * (np.abs(u) + np.abs(v))
    bound[..., i], bound[..., j] = b, b
    return y, bound


def rms_norm(h, w, eps=1e-6):
    """y of rows h [.., C]: (y, bound).  The mean square is a sum of at most 128 roundings a term
    (a thread's values, shuffles, warps), of which 1/rstd takes half; rsqrt and two products add a
    few: 80 EPS of |y|."""
    h, w = _f64(h), _f64(w)
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w
    return y, 80 * EPS * np.abs(y)


def rms_norm_backward(h, w, dy, dres=None, eps=1e-6):
    """(dx, dw) and their bounds: the sums as for rms_norm (128 roundings a term, on the absolute
    values), dw one rounding a row and 256 for the joins of threads and CTAs."""
    h, w, dy = _f64(h), _f64(w), _f64(dy)
    rstd = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, p = h * rstd, dy * w
    dx = rstd * (p - n * (p * n).mean(-1, keepdims=True))
    size = rstd * (np.abs(p) + np.abs(n) * np.abs(p * n).mean(-1, keepdims=True))
    if dres is not None:
        dx = dx + _f64(dres)
        size = size + np.abs(_f64(dres))
    axes = tuple(range(h.ndim - 1))
    rows = int(np.prod(h.shape[:-1]))
    return ((dx, (dy * n).sum(axes)),
            (400 * EPS * size, (rows + 400) * EPS * np.abs(dy * n).sum(axes)))
