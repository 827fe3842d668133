"""GPU parity of rotary positions (``la_rotary``) against the fp64 oracle.

Tolerance, element by element: the oracle's bound (8 half steps of fp32 of |u| + |v|) plus half a
step of the output's type.  Values that pass through are copies and must match exactly.
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


def heads(x, d):
    """Token-major [B, T, H*d] as head-major fp64 [B, H, T, d]."""
    return np.moveaxis(f64(x).reshape(*x.shape[:2], -1, d), 2, 1)


def rand(dtype, *shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


# (B, T, H, Hk, d, r): vectors and scalars (r not a multiple of 16, d not of 8), one head, shared
# key heads, more key than query heads, parts of a head, a lone last vector (d - r = 8, 12), tokens
# enough that a warp is one token whose threads share the angles
CASES = [(1, 1, 1, 1, 64, 64), (2, 5, 3, 1, 64, 32), (1, 37, 16, 4, 128, 128), (3, 9, 5, 5, 128, 64),
         (1, 20, 1, 7, 64, 16), (2, 7, 2, 2, 24, 16), (1, 6, 4, 2, 64, 24), (1, 11, 3, 2, 10, 6),
         (2, 3, 2, 1, 7, 2), (1, 4, 9, 0, 256, 64), (1, 3, 33, 8, 80, 80), (1, 2, 2, 1, 512, 512),
         (2, 9, 3, 2, 36, 24), (2, 1300, 6, 2, 128, 64), (1, 2500, 5, 3, 64, 32), (1, 2400, 1, 1, 128, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_matches_oracle(la, dtype, case, interleaved):
    B, T, H, Hk, d, r = case
    q = rand(dtype, B, T, H * d, seed=T)
    k = rand(dtype, B, T, Hk * d, seed=T + 1) if Hk else None
    freqs, _ = la.rotary_frequencies(r)
    pos = np.arange(1000, 1000 + T) + np.zeros((B, 1))
    got = la.rotary(q, k, freqs=freqs, d=d, start=1000, scale=1.25, interleaved=interleaved)
    la.check_status()
    for x, y in zip((q, k), got if Hk else (got,)):
        ref, b = L.rotary(heads(x, d), pos, f64(freqs), 1.25, interleaved)
        close(y, ref, b)
        np.testing.assert_array_equal(f64(y)[..., r:], ref[..., r:])
        # backwards from the head-major rows to the projections' layout
        dy = rand(dtype, *y.shape, seed=T + 2)
        dx = la.rotary_backward(dy, freqs=freqs, start=1000, scale=1.25, interleaved=interleaved, token_major=True)
        la.check_status()
        assert dx.shape == x.shape
        ref, b = L.rotary(f64(dy), pos, f64(freqs), 1.25, interleaved, transpose=True)
        close(dx, *(np.moveaxis(v, 1, 2).reshape(dx.shape) for v in (ref, b)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("start", [0, 262143, 2 ** 31 - 40, -2 ** 31])
def test_rotary_far_positions(la, dtype, start):
    """Angles of far positions: fp64 keeps them to 2^-20 of a turn (freqs of a power of two times
    their exact values are formed the same way in the oracle)."""
    q = rand(dtype, 1, 33, 4 * 64, seed=3)
    freqs = torch.tensor([2.0 ** -j for j in range(16)], dtype=torch.float64, device="cuda")
    y = la.rotary(q, freqs=freqs, d=64, start=start)
    la.check_status()
    pos = start + np.arange(33, dtype=np.float64)[None]
    ref, b = L.rotary(heads(q, 64), pos, f64(freqs))
    # the product with 1 / (2 pi) and its own rounding: two half steps of fp64 of the angle
    x = np.abs(heads(q, 64))
    far = 4 * 2.0 ** -53 * abs(float(pos.max() if start > 0 else start))
    close(y, ref, b + far * (x + np.roll(x, 16, -1) + np.roll(x, -16, -1)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("r", [64, 32, 24])
def test_rotary_positions_packed_and_step(la, interleaved, r):
    """Packed sequences (positions that restart) and single tokens at their own positions, also
    negative and repeated ones."""
    d, H, Hk = 64, 4, 2
    freqs, _ = la.rotary_frequencies(r, base=500000.0)
    pos = torch.tensor([0, 1, 2, 0, 1, 7, 7, -3, 100000, 5], dtype=torch.int32, device="cuda")
    q, k = rand(torch.bfloat16, 1, 10, H * d, seed=1), rand(torch.bfloat16, 1, 10, Hk * d, seed=2)
    yq, yk = la.rotary(q, k, freqs=freqs, d=d, positions=pos[None], interleaved=interleaved)
    sq, sk = la.rotary_step(q[0], k[0], freqs=freqs, d=d, positions=pos, interleaved=interleaved)
    la.check_status()
    for x, y, s in ((q, yq, sq), (k, yk, sk)):
        close(y, *L.rotary(heads(x, d), pos.cpu().numpy()[None], f64(freqs), 1.0, interleaved))
        assert torch.equal(s, y[0].transpose(0, 1))


@pytest.mark.parametrize("r", [128, 64, 30])
def test_rotary_in_place_and_layouts(la, r):
    B, T, H, d = 2, 19, 3, 128
    freqs, _ = la.rotary_frequencies(r)
    x = rand(torch.bfloat16, B, T, H * d, seed=8)
    want = la.rotary(x, freqs=freqs, d=d, start=5)
    rows = x.view(B, T, H, d).transpose(1, 2).contiguous()
    assert torch.equal(la.rotary(rows, freqs=freqs, start=5), want)
    k = rows[:, :1].contiguous()
    got = la.rotary(rows, k, freqs=freqs, start=5, in_place=True)
    la.check_status()
    assert got[0].data_ptr() == rows.data_ptr() and got[1].data_ptr() == k.data_ptr()
    assert torch.equal(rows, want) and torch.equal(k, want[:, :1])
    dx = rand(torch.bfloat16, B, T, H * d, seed=9)
    a = la.rotary_backward(dx, freqs=freqs, d=d, start=5, token_major=True)
    b = la.rotary_backward(dx.view(B, T, H, d).transpose(1, 2).contiguous(), freqs=freqs, start=5, token_major=True)
    c = la.rotary_backward(dx.clone(), freqs=freqs, d=d, start=5, token_major=True, in_place=True)
    assert torch.equal(a, b) and torch.equal(a, c)


def test_rotary_empty_and_refusals(la):
    freqs, _ = la.rotary_frequencies(64)
    y = la.rotary(torch.zeros(2, 0, 128, device="cuda"), freqs=freqs, d=64)
    assert y.shape == (2, 2, 0, 64)
    x = torch.zeros(1, 4, 128, device="cuda")
    lib, p = la.library(), (lambda t: t.data_ptr())
    # the same buffer in another layout would be a race
    st = lib.la_rotary(0, 1, 4, 2, 0, 64, 64, p(x), None, p(freqs), None, 0, 1.0, p(x), None, la.ROT_X_TOKENS, None)
    assert st == 1
    st = lib.la_rotary(0, 1, 4, 2, 2, 64, 64, p(x), p(x), p(freqs), None, 0, 1.0, p(x), p(x), 0, None)
    assert st == 1   # q and k in one buffer
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.rotary(x, freqs=freqs.cpu(), d=64)
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.rotary(torch.zeros(513, device="cuda")[1:].view(1, 4, 128), freqs=freqs, d=64)
    with pytest.raises(la.LaError, match="UNSUPPORTED"):
        la.rotary(torch.zeros(1, 1, 1024, device="cuda"), freqs=freqs, d=1024)
    la.check_status()


def test_rotary_offsets_beyond_32_bits(la):
    T, H, d = 2 ** 31 // 512 + 33, 4, 128
    q = torch.empty(1, T, H * d, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    freqs, _ = la.rotary_frequencies(d)
    y = la.rotary(q, freqs=freqs, d=d)
    tail = la.rotary(q[:, -40:].contiguous(), freqs=freqs, d=d, start=T - 40)
    la.check_status()
    assert torch.equal(y[:, :, -40:], tail)
    back = la.rotary_backward(y, freqs=freqs, token_major=True)
    assert torch.equal(back[:, -40:], la.rotary_backward(tail, freqs=freqs, start=T - 40, token_major=True))
