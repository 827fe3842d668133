"""Refusals and host-side parts of the operators around the attention, without a GPU.

The argument checks run on the host before anything is launched: with null or host pointers
every call below answers with a status and touches no device.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def la():
    from gated_delta_rule_attention_b200 import build
    build.build()
    import gated_delta_rule_attention_b200 as m
    m.library()
    return m


def test_scan_refusals(la):
    lib = la.library()

    def scan(dtype=1, B=1, T=8, C=8, flags=0):
        return lib.la_linear_scan(dtype, B, T, C, None, None, None, None, None, flags, None)

    for bad in (dict(dtype=2), dict(B=0), dict(T=-1), dict(C=0), dict(flags=4), dict(), dict(T=0),
                dict(B=2 ** 31 - 1, T=2 ** 31 - 1, C=2 ** 31 - 1)):
        assert scan(**bad) == INVALID
    assert lib.la_linear_scan_step(1, 4, 8, None, None, None, None, 1, None) == INVALID   # no INIT flag here
    assert lib.la_linear_scan_step(1, 0, 8, None, None, None, None, 0, None) == INVALID

    def packed(N=1, T=8, C=8):
        return lib.la_linear_scan_varlen(1, N, T, C, None, None, None, None, None, 0, None, 0, None)

    for bad in (dict(), dict(N=0), dict(N=1 << 29), dict(T=2 ** 31 - 1)):
        assert packed(**bad) == INVALID
    back = [None] * 9
    assert lib.la_linear_scan_backward(1, 1, 0, 8, *back, 0, None, 0, None) == INVALID
    assert lib.la_linear_scan_backward(1, 1, 8, 8, *back, 0, None, 0, None) == INVALID
    assert lib.la_linear_scan_backward(1, 1, 8, 8, *back, 1, None, 0, None) == INVALID


def test_workspace_sizes(la):
    lib = la.library()
    assert lib.la_linear_scan_varlen_workspace_size(0) == 0
    assert lib.la_linear_scan_varlen_workspace_size(33) == 4 * 256
    assert lib.la_linear_scan_backward_workspace_size(2, 65, 100) == 4 * 2 * 3 * 100
    assert lib.la_linear_scan_backward_workspace_size(2, 0, 100) == 0
    assert lib.la_rms_norm_backward_workspace_size(1, 1, 3, 100) == 4 * 3 * 100
    assert lib.la_rms_norm_backward_workspace_size(1, 1, 10 ** 6, 100) <= 4 * 100 * 148 * 8
    assert lib.la_rms_norm_backward_workspace_size(1, 1, 3, 20000) == 0


def test_rotary_refusals(la):
    lib = la.library()

    def rot(dtype=1, B=1, T=4, Hq=2, Hk=1, d=64, r=64, flags=0):
        return lib.la_rotary(dtype, B, T, Hq, Hk, d, r, None, None, None, None, 0, 1.0, None, None, flags, None)

    for bad in (dict(), dict(dtype=3), dict(B=0), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(r=0), dict(r=7),
                dict(r=66), dict(flags=16)):
        assert rot(**bad) == INVALID
    assert rot(d=640, r=64) == UNSUPPORTED
    assert rot(T=0) == OK


def test_norm_refusals(la):
    lib = la.library()

    def norm(dtype=1, B=1, H=1, T=4, C=128, eps=1e-6, group=0, flags=0, res=None):
        return lib.la_rms_norm(dtype, B, H, T, C, None, res, None, eps, None, None, None, group, flags, None)

    for bad in (dict(), dict(dtype=2), dict(B=0), dict(H=0), dict(T=-1), dict(C=0), dict(eps=-1.0),
                dict(eps=math.nan), dict(group=128), dict(group=64, flags=1), dict(group=128, C=192, flags=1),
                dict(flags=2), dict(H=2, res=ctypes.c_void_p(16))):
        assert norm(**bad) == INVALID, bad
    assert norm(C=16385) == UNSUPPORTED
    assert norm(T=0) == OK
    assert lib.la_rms_norm_backward(1, 1, 1, 4, 128, *[None] * 2, 1e-6, *[None] * 5, 0, None) == INVALID
    assert lib.la_rms_norm_backward(1, 1, 1, 4, 17000, *[None] * 2, 1e-6, *[None] * 5, 0, None) == UNSUPPORTED


def test_host_pointers_are_rejected(la):
    lib = la.library()
    buf = np.zeros(1 << 14, dtype=np.float32)
    p = ctypes.c_void_p((buf.ctypes.data + 15) // 16 * 16)
    assert lib.la_linear_scan(0, 1, 4, 8, p, p, p, p, None, 0, None) == INVALID
    assert lib.la_linear_scan_step(0, 1, 8, p, p, p, p, 0, None) == INVALID
    assert lib.la_rotary(0, 1, 4, 1, 0, 64, 64, p, None, p, None, 0, 1.0, p, None, 0, None) == INVALID
    assert lib.la_rms_norm(0, 1, 1, 4, 64, p, None, p, 1e-6, None, p, None, 0, 0, None) == INVALID


def test_python_checks(la):
    x, g = torch.zeros(1, 4, 8), torch.zeros(1, 4, 8)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        la.linear_scan(x.half(), g)
    with pytest.raises(TypeError, match="gate"):
        la.linear_scan(x, g.double())
    with pytest.raises(ValueError, match="gate"):
        la.linear_scan(x, g[:, :3])
    with pytest.raises(ValueError, match="contiguous"):
        la.linear_scan(torch.zeros(1, 8, 4).transpose(1, 2), g)
    with pytest.raises(ValueError, match="init_state"):
        la.linear_scan(x, g, init_state=True)
    with pytest.raises(ValueError, match="two entries"):
        la.linear_scan_varlen(x[0], g[0], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="checkpoints"):
        la.linear_scan_backward(x, g, x, checkpoints=torch.zeros(1, 2, 8))
    f, _ = la.rotary_frequencies(8, device="cpu")
    with pytest.raises(ValueError, match="needs d"):
        la.rotary(x, freqs=f)
    with pytest.raises(ValueError, match="layout"):
        la.rotary(torch.zeros(1, 2, 4, 8), x, freqs=f, d=8)
    with pytest.raises(TypeError, match="freqs"):
        la.rotary(x, freqs=f.float(), d=8)
    with pytest.raises(ValueError, match="in_place"):
        la.rotary(x, freqs=f, d=8, in_place=True)
    with pytest.raises(ValueError, match="32 bits"):
        la.rotary(x, freqs=f, d=8, start=2 ** 31)
    with pytest.raises(ValueError, match="heads"):
        la.rotary(torch.empty(1, 1, 2 ** 33, device="meta"), freqs=f[:1], d=2)
    with pytest.raises(ValueError, match="positions"):
        la.rotary_step(x[0], freqs=f, d=8, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="group"):
        la.rms_norm(x, torch.ones(8), fp8=True, group=128)
    with pytest.raises(ValueError, match="fp8"):
        la.rms_norm(x, torch.ones(8), group=8)
    with pytest.raises(ValueError, match="residual"):
        la.rms_norm(x, torch.ones(8), residual_out=x)


def test_rotary_frequencies(la):
    plain, s = la.rotary_frequencies(64, device="cpu")
    assert s == 1.0 and plain.dtype == torch.float64
    np.testing.assert_allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    lin, _ = la.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(lin, plain / 4, rtol=1e-15)
    ntk, _ = la.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == plain[0] and float(ntk[-1] / plain[-1]) == pytest.approx(0.25)
    yarn, s = la.rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu")
    assert s == pytest.approx(0.1 * math.log(4) + 1)
    turns = plain * 4096 / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], plain[turns > 32])
    np.testing.assert_allclose(yarn[turns < 1], plain[turns < 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (yarn[mid] < plain[mid]).all() and (yarn[mid] > plain[mid] / 4).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=2, scaling="ntk"),
                dict(rotary_dim=8, scaling="yarn"), dict(rotary_dim=8, scaling="other"),
                dict(rotary_dim=8, factor=0.0)):
        with pytest.raises(ValueError):
            la.rotary_frequencies(**bad, device="cpu")
