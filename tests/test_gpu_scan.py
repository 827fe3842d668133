"""GPU parity of the gated linear recurrence (``la_linear_scan*``) against the fp64 oracle.

Tolerances are the oracle's bounds of what fp32 arithmetic may add (see ``oracle/layer.py``),
element by element, plus half a step of the output's type: 2^-8 of the value for bf16, 2^-24 for
fp32.  The oracle gets the exact values the GPU receives.
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
    off = np.abs(y - ref) - (bound * (1 + half) + half * np.abs(ref))
    bad = ~(off <= 0)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside; worst by {off.max():.3e} at {np.unravel_index(off.argmax(), off.shape)}"


def inputs(dtype, *shape, seed=0, long_memory=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda").to(dtype)
    if long_memory:
        gate = 1 - torch.rand(*shape, generator=g, device="cuda") * 1e-3
    else:
        gate = torch.rand(*shape, generator=g, device="cuda") ** 0.3
    return x, gate, torch.randn(shape[0], shape[-1], generator=g, device="cuda")


# one row, the edges of a thread's, a tile's and a checkpoint's rows, several steps of clusters;
# channels odd, even, multiples of 4, one, and not filling a block
SHAPES = [(1, 1, 1), (2, 1, 64), (1, 7, 5), (3, 8, 12), (2, 9, 66), (1, 31, 64), (2, 32, 7), (1, 33, 128),
          (1, 127, 40), (2, 128, 4), (1, 129, 130), (1, 511, 20), (2, 640, 100), (1, 2049, 33), (1, 3001, 16),
          (5, 300, 2)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("blend,init", [(False, False), (True, True)])
def test_scan_matches_oracle(la, dtype, shape, blend, init):
    x, gate, h0 = inputs(dtype, *shape, seed=sum(shape))
    start = h0.clone()
    h, state = la.linear_scan(x, gate, state=h0 if init else None, blend=blend)
    la.check_status()
    rh, rs, b = L.linear_scan(f64(x), f64(gate), f64(start) if init else None, blend)
    close(h, rh, b)
    close(state, rs, b[:, -1])
    if init:
        assert state.data_ptr() == h0.data_ptr()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("blend,init", [(False, True), (True, False)])
def test_scan_backward_matches_oracle(la, dtype, shape, blend, init):
    x, gate, h0 = inputs(dtype, *shape, seed=1 + sum(shape))
    dh, _, ds = inputs(dtype, *shape, seed=2 + sum(shape))
    start = h0 if init else None
    h, state, kept = la.linear_scan(x, gate, state=h0.clone() if init else None, blend=blend, checkpoints=True)
    got = la.linear_scan_backward(x, gate, dh, checkpoints=kept, dstate=ds if init else None, blend=blend,
                                  need_dstate0=True)
    again = la.linear_scan_backward(x, gate, dh, state0=start, dstate=ds if init else None, blend=blend,
                                    need_dstate0=True)
    la.check_status()
    # the kept states: in front of rows 0, 32, ..
    rh, _, b = L.linear_scan(f64(x), f64(gate), None if start is None else f64(start), blend)
    first = np.zeros_like(rh[:, :1]) if start is None else f64(start)[:, None]
    at = slice(31, shape[1] - 1, 32)
    close(kept, np.concatenate([first, rh[:, at]], 1), np.concatenate([0 * first, b[:, at]], 1))
    refs, bounds = L.linear_scan_backward(f64(x), f64(gate), f64(dh), None if start is None else f64(start),
                                          f64(ds) if init else None, blend)
    for y, z, ref, bound in zip(got, again, refs, bounds):
        close(y, ref, bound)
        assert torch.equal(y, z)   # the states formed again are the same bits


@pytest.mark.parametrize("shape", [(1, 70000, 8), (2, 20000, 20), (1, 9000, 260)])
def test_scan_long_memory(la, shape):
    """Gates next to 1 over many cluster steps: nothing decays, so every join counts."""
    x, gate, h0 = inputs(torch.float32, *shape, seed=7, long_memory=True)
    dh = torch.randn_like(x)
    h, state, kept = la.linear_scan(x, gate, state=h0.clone(), checkpoints=True)
    got = la.linear_scan_backward(x, gate, dh, checkpoints=kept, need_dstate0=True)
    la.check_status()
    rh, rs, b = L.linear_scan(f64(x), f64(gate), f64(h0))
    close(h, rh, b)
    close(state, rs, b[:, -1])
    refs, bounds = L.linear_scan_backward(f64(x), f64(gate), f64(dh), f64(h0))
    for y, ref, bound in zip(got, refs, bounds):
        close(y, ref, bound)


@pytest.mark.parametrize("cols", [8, 16, 37 * 64, 149 * 64, 600 * 64 + 4])
def test_scan_every_cluster_width(la, cols):
    """Few and many columns: every width of a cluster, and further waves of them."""
    x, gate, h0 = inputs(torch.bfloat16, 1, 1200, cols, seed=cols)
    h, state = la.linear_scan(x, gate, state=h0.clone(), blend=True)
    la.check_status()
    some = torch.arange(0, cols, max(1, cols // 50), device="cuda")
    rh, rs, b = L.linear_scan(f64(x[:, :, some]), f64(gate[:, :, some]), f64(h0[:, some]), True)
    close(h[:, :, some], rh, b)
    close(state[:, some], rs, b[:, -1])


def test_scan_is_the_same_bits_and_splits(la):
    x, gate, h0 = inputs(torch.float32, 2, 1000, 96, seed=3)
    a = la.linear_scan(x, gate, state=h0.clone())
    b = la.linear_scan(x, gate, state=h0.clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    state = h0.clone()
    parts = [la.linear_scan(x[:, i:j].contiguous(), gate[:, i:j].contiguous(), state=state)[0]
             for i, j in ((0, 1), (1, 400), (400, 1000))]
    rh, _, bound = L.linear_scan(f64(x), f64(gate), f64(h0))
    close(torch.cat(parts, 1), rh, 2 * bound)


def test_scan_gates_of_zero_and_one(la):
    x, gate, h0 = inputs(torch.float32, 1, 700, 64, seed=4)
    gate[:, ::3] = 1.0
    gate[:, 100:140] = 0.0
    gate[:, 600:] = 0.0
    for blend in (False, True):
        h, state, kept = la.linear_scan(x, gate, state=h0.clone(), blend=blend, checkpoints=True)
        dh = torch.randn_like(x)
        got = la.linear_scan_backward(x, gate, dh, checkpoints=kept, blend=blend, need_dstate0=True)
        la.check_status()
        rh, rs, b = L.linear_scan(f64(x), f64(gate), f64(h0), blend)
        close(h, rh, b)
        refs, bounds = L.linear_scan_backward(f64(x), f64(gate), f64(dh), f64(h0), None, blend)
        for y, ref, bound in zip(got, refs, bounds):
            close(y, ref, bound)


def test_scan_nan_reaches_what_follows_it_alone(la):
    x, gate, _ = inputs(torch.float32, 1, 400, 64, seed=5)
    clean, _ = la.linear_scan(x, gate)
    x[0, 150, 10] = float("nan")
    h, state = la.linear_scan(x, gate)
    la.check_status()
    assert torch.isnan(h[0, 150:, 10]).all() and torch.isnan(state[0, 10])
    h[0, 150:, 10] = clean[0, 150:, 10]
    assert torch.equal(h, clean)


def test_scan_empty(la):
    x = torch.zeros(2, 0, 8, device="cuda")
    h, state = la.linear_scan(x, x)
    assert h.shape == (2, 0, 8) and float(state.abs().max()) == 0.0
    keep = torch.ones(2, 8, device="cuda")
    _, state = la.linear_scan(x, x, state=keep)
    assert torch.equal(state, torch.ones_like(keep))


LENGTHS = [[5], [1], [0, 0, 3], [65, 0, 1, 64, 130, 63, 200, 2], [1] * 40, [300, 1, 1, 0, 70, 1000, 0], [2500, 31, 33]]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("C", [64, 40, 50, 7])
@pytest.mark.parametrize("init", [False, True])
def test_scan_varlen_matches_oracle(la, dtype, lengths, C, init):
    T, N = sum(lengths), len(lengths)
    x, gate, _ = inputs(dtype, T, C, seed=T + C)
    state = torch.randn(N, C, device="cuda") if init else None
    start = None if state is None else f64(state)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    h, last = la.linear_scan_varlen(x, gate, cu, state=state, blend=init)
    la.check_status()
    rh, rs, b = L.linear_scan_packed(f64(x), f64(gate), cu.tolist(), start, init)
    close(h, rh, b)
    ends = np.array([b[cu[s + 1].item() - 1] if lengths[s] else 0 * b[0] for s in range(N)])
    close(last, rs, ends)


def test_scan_varlen_rows_of_no_sequence_stay(la):
    x, gate, _ = inputs(torch.bfloat16, 300, 64, seed=9)
    x[:20] = float("nan")
    x[250:] = float("nan")
    cu = torch.tensor([20, 100, 100, 250], dtype=torch.int32, device="cuda")
    h = torch.full_like(x, 5.0)
    _, state = la.linear_scan_varlen(x, gate, cu, h=h)
    la.check_status()
    assert (h[:20] == 5).all() and (h[250:] == 5).all()
    rh, rs, b = L.linear_scan_packed(f64(x), f64(gate), cu.tolist())
    close(h[20:250], rh[20:250], b[20:250])
    assert float(state[1].abs().max()) == 0.0


def test_scan_varlen_nan_stays_in_its_sequence(la):
    x, gate, _ = inputs(torch.float32, 900, 36, seed=10)
    cu = torch.tensor([0, 100, 101, 333, 650, 900], dtype=torch.int32, device="cuda")
    state = torch.randn(5, 36, device="cuda")
    clean, ends = la.linear_scan_varlen(x, gate, cu, state=state.clone())
    x[50] = float("nan")
    x[640] = float("inf")
    x[645] = float("-inf")
    h, last = la.linear_scan_varlen(x, gate, cu, state=state.clone())
    la.check_status()
    for s in (1, 2, 4):
        assert torch.equal(h[cu[s]:cu[s + 1]], clean[cu[s]:cu[s + 1]]) and torch.equal(last[s], ends[s])
    assert torch.isnan(last[0]).all() and torch.isnan(last[3]).all()


def test_scan_varlen_many_sequences_in_place(la):
    """More sequences than rows of a tile, the state read and written in place, against dense calls."""
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 60, (400,), generator=g).tolist()
    T, C = sum(lengths), 128
    x, gate, _ = inputs(torch.float32, T, C, seed=11)
    state = torch.randn(400, C, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    rh, rs, b = L.linear_scan_packed(f64(x), f64(gate), cu.tolist(), f64(state))
    h, last = la.linear_scan_varlen(x, gate, cu, state=state)
    la.check_status()
    assert last.data_ptr() == state.data_ptr()
    close(h, rh, b)


@pytest.mark.parametrize("C", [192, 1024, 101])
def test_scan_varlen_sees_what_the_stream_wrote(la, C):
    """Inputs, offsets and states written by kernels right in front of the call, in turn, with nothing
    waited for in between: the same bits as of calls by themselves."""
    T, N, kinds = 6000, 37, 3
    g = torch.Generator().manual_seed(C)
    given, want = [], []
    for i in range(kinds):
        x, gate, _ = inputs(torch.bfloat16, T, C, seed=C + i)
        cuts = torch.randint(0, T + 1, (N - 1,), generator=g).sort().values.tolist()
        cu = torch.tensor([0, *cuts, T], dtype=torch.int32, device="cuda")
        given.append((x, gate, cu, torch.randn(N, C, device="cuda")))
        state = given[i][3].clone()
        torch.cuda.synchronize()
        want.append((la.linear_scan_varlen(x, gate, cu, state=state)[0], state))
        torch.cuda.synchronize()
    x, gate, cu, state = (torch.empty_like(t) for t in given[0])
    got = []
    for i in range(30):
        for to, t in zip((x, gate, cu, state), given[i % kinds]):
            to.copy_(t)
        h, _ = la.linear_scan_varlen(x, gate, cu, state=state)
        got.append((h, state.clone()))
    la.check_status()
    for i, (h, last) in enumerate(got):
        assert torch.equal(h, want[i % kinds][0]) and torch.equal(last, want[i % kinds][1]), i


def test_scan_state_in_place_over_clusters(la):
    """The state read and written in place by calls that split the time over a cluster."""
    x, gate, _ = inputs(torch.float32, 2, 700, 64, seed=21)
    h0 = torch.randn(2, 64, device="cuda")
    want, end = la.linear_scan(x, gate, state=h0.clone())
    for _ in range(50):
        state = h0.clone()
        h, _ = la.linear_scan(x, gate, state=state)
        assert torch.equal(h, want) and torch.equal(state, end)
    la.check_status()


def test_scan_varlen_bad_offsets_are_reported(la):
    x, gate, _ = inputs(torch.bfloat16, 100, 64, seed=1)
    for bad in ([0, 60, 40, 500], [-5, 50, 100, 100], [0, 200, 300, 400]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        la.linear_scan_varlen(x, gate, cu)
        with pytest.raises(la.LaError, match="INVALID_ARG"):
            la.check_status()
    la.check_status()


def test_scan_varlen_empty_batch(la):
    x = torch.zeros(0, 8, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    _, state = la.linear_scan_varlen(x, x, cu)
    la.check_status()
    assert float(state.abs().max()) == 0.0
    keep = torch.ones(3, 8, device="cuda")
    la.linear_scan_varlen(x, x, cu, state=keep)
    la.check_status()
    assert torch.equal(keep, torch.ones_like(keep))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,C", [(1, 1), (3, 5), (2, 64), (7, 130), (256, 1000)])
@pytest.mark.parametrize("blend", [False, True])
def test_scan_step_continues_the_scan(la, dtype, N, C, blend):
    x, gate, h0 = inputs(dtype, N, 12, C, seed=N + C)
    state = h0.clone()
    _, state = la.linear_scan(x[:, :9].contiguous(), gate[:, :9].contiguous(), state=state, blend=blend)
    rh, rs, b = L.linear_scan(f64(x), f64(gate), f64(h0), blend)
    for t in range(9, 12):
        h = la.linear_scan_step(x[:, t].contiguous(), gate[:, t].contiguous(), state, blend=blend)
        la.check_status()
        close(h, rh[:, t], b[:, t])
        close(state, rs if t == 11 else rh[:, t], b[:, t])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_scan_takes_tensors_that_start_anywhere(la, dtype, off):
    """Parts of larger tensors: the same result (joins in another order) as from aligned copies."""
    B, T, C = 1, 200, 64
    x, gate, h0 = inputs(dtype, B, T, C, seed=off)

    def moved(t):
        big = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        big[off:off + t.numel()] = t.reshape(-1)
        return big[off:off + t.numel()].view(t.shape)

    rh, rs, b = L.linear_scan(f64(x), f64(gate), f64(h0))
    h, state, kept = la.linear_scan(moved(x), moved(gate), state=moved(h0), h=moved(torch.zeros_like(x)), checkpoints=True)
    got = la.linear_scan_backward(moved(x), moved(gate), moved(x), checkpoints=moved(kept), dstate=moved(h0),
                                  need_dstate0=True)
    one = moved(h0)
    s1 = la.linear_scan_step(moved(x[:, 0]), moved(gate[:, 0]), one, h=moved(torch.zeros_like(x[:, 0])))
    la.check_status()
    close(h, rh, b)
    close(state, rs, b[:, -1])
    close(s1, rh[:, 0], b[:, 0])
    refs, bounds = L.linear_scan_backward(f64(x), f64(gate), f64(x), f64(h0), f64(h0))
    for y, ref, bound in zip(got, refs, bounds):
        close(y, ref, bound)


def test_scan_refuses_overlaps_and_host_tensors(la):
    x = torch.zeros(1, 8, 8, device="cuda")
    gate = torch.zeros_like(x)
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.linear_scan(x, gate, h=x)
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.linear_scan_step(x[0], gate[0], gate[0])
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.linear_scan(x, torch.zeros(1, 8, 8))          # a gate on the host
    with pytest.raises(la.LaError, match="INVALID_ARG"):
        la.linear_scan_varlen(x[0], gate[0], torch.tensor([0, 8], dtype=torch.int32), h=torch.zeros_like(x[0]))
    la.check_status()


def test_scan_gradient_against_differences(la):
    """The backward kernel against differences of the forward kernel, in fp32: a step of 2^-6 along
    a direction; the loss is linear in x and in h_0 (exact but for rounding) and a polynomial in
    the gates (truncation error of the second order, 2^-12 times the third derivative)."""
    x, gate, h0 = inputs(torch.float32, 2, 40, 12, seed=21)
    gate = 0.2 + 0.6 * gate
    dh = torch.randn_like(x)
    ds = torch.randn_like(h0)
    e = 2.0 ** -6

    def loss(x, gate, h0):
        h, s = la.linear_scan(x, gate, state=h0.clone(), blend=True)
        return float((h.double() * dh).sum() + (s.double() * ds).sum())

    dx, dg, d0 = la.linear_scan_backward(x, gate, dh, state0=h0, dstate=ds, blend=True)
    for i, (t, grad, tol) in enumerate(((x, dx, 2e-3), (gate, dg, 2e-2), (h0, d0, 2e-3))):
        d = torch.randn_like(t) * (0.2 if i == 1 else 1.0)
        args = [[x, gate, h0], [x, gate, h0]]
        args[0][i], args[1][i] = t + e * d, t - e * d
        num = (loss(*args[0]) - loss(*args[1])) / (2 * e)
        assert num == pytest.approx(float((grad.double() * d).sum()), rel=tol, abs=tol * float((grad.double() * d).norm()))


@pytest.mark.parametrize("C", [64, 34, 7])
@pytest.mark.parametrize("blend", [False, True])
def test_scan_backward_without_the_gates(la, C, blend):
    x, gate, h0 = inputs(torch.bfloat16, 2, 150, C, seed=C)
    want = la.linear_scan_backward(x, gate, x, state0=h0, blend=blend)
    got = la.linear_scan_backward(x, gate, x, state0=h0, blend=blend, need_dgate=False, need_dstate0=False)
    la.check_status()
    assert got[1] is None and got[2] is None and torch.equal(got[0], want[0])


@pytest.mark.parametrize("C", [4096, 4094, 4095])
def test_scan_offsets_beyond_32_bits(la, C):
    """More than 2^31 elements: closed gates 500 rows before the end make the last rows those of a
    short call on them."""
    T = 2 ** 31 // C + 700
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    gate = torch.empty(1, T, C, device="cuda").uniform_(0.5, 1)
    gate[:, T - 500] = 0
    h, state, kept = la.linear_scan(x, gate, checkpoints=True)
    dx, dgate, _ = la.linear_scan_backward(x, gate, x, checkpoints=kept)
    tx, tg = x[:, T - 500:].contiguous(), gate[:, T - 500:].contiguous()
    rh, rs, b = L.linear_scan(f64(tx), f64(tg))
    refs, bounds = L.linear_scan_backward(f64(tx), f64(tg), f64(tx))
    la.check_status()
    close(h[:, T - 500:], rh, b)
    close(state, rs, b[:, -1])
    close(dx[:, T - 500:], refs[0], bounds[0])
    close(dgate[:, T - 499:], refs[1][:, 1:], bounds[1][:, 1:])
    # and the first rows, whose gradients end the reverse walk
    gate[:, 500] = 0
    dx, _, _ = la.linear_scan_backward(x, gate, x, need_dgate=False)
    refs, bounds = L.linear_scan_backward(f64(x[:, :501]), f64(gate[:, :501]), f64(x[:, :501]))
    close(dx[:, :500], refs[0][:, :500], bounds[0][:, :500])
