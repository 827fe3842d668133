"""The operators around the attention as they are used together, on other streams, in captured
graphs, and by two threads at once."""
import threading

import numpy as np
import pytest
import torch

import oracle
from oracle import layer as L
from parity_util import TOL, f64, slice_rel_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    import gated_delta_rule_attention_b200 as m
    m.library()
    return m


def rand(dtype, *shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def heads(x, d):
    return np.moveaxis(f64(x).reshape(*x.shape[:2], -1, d), 2, 1)


def test_constant_decay_layer_prefill_then_decode(la):
    """Norm with residual -> projections -> rotary -> constant-decay attention -> norm of the heads,
    a prompt and then a token of it, against the oracles on the same bf16 values."""
    B, T, H, d, dt = 2, 90, 2, 128, torch.bfloat16
    C = H * d
    x, res = rand(dt, B, T + 1, C, seed=1), rand(dt, B, T + 1, C, seed=2)
    w, wh = 1 + 0.2 * rand(torch.float32, C, seed=3), 1 + 0.2 * rand(torch.float32, d, seed=4)
    proj = [rand(dt, C, C, seed=5 + i) * C ** -0.5 for i in range(3)]
    gamma = torch.tensor([0.9, 0.99], device="cuda")
    freqs, _ = la.rotary_frequencies(d)
    y, h = la.rms_norm(x, w, residual=res)
    q, k, v = (y @ p for p in proj)
    rq, rk = la.rotary(q[:, :T].contiguous(), k[:, :T].contiguous(), freqs=freqs, d=d, scale=d ** -0.25)
    vh = v[:, :T].reshape(B, T, H, d).transpose(1, 2).contiguous()
    o, S, _ = la.prefill(rq, rk, vh, mode=la.MODE_RETNET, gate=gamma)
    out = la.rms_norm_heads(o, wh)
    # the next token
    at = torch.full((B,), T, dtype=torch.int32, device="cuda")
    sq, sk = la.rotary_step(q[:, T].contiguous(), k[:, T].contiguous(), freqs=freqs, d=d, positions=at,
                            scale=d ** -0.25)
    keep = S.clone()
    o1, S1, _ = la.decode_step(sq, sk, v[:, T].reshape(B, H, d).contiguous(), mode=la.MODE_RETNET, state=S, gate=gamma)
    out1 = la.rms_norm_heads(o1.unsqueeze(2), wh)
    la.check_status()
    ry, _ = L.rms_norm(f64(h), f64(w))
    assert slice_rel_err(f64(y), ry) < TOL[dt]
    pos = np.arange(T + 1)[None] + np.zeros((B, 1))
    fq, fk = (L.rotary(heads(t, d), pos, f64(freqs), d ** -0.25)[0] for t in (q, k))
    for got, step, ref in ((rq, sq, fq), (rk, sk, fk)):
        assert slice_rel_err(f64(got), ref[:, :, :T]) < 2.0 ** -7
        assert slice_rel_err(f64(step), ref[:, :, T]) < 2.0 ** -7
    g = np.broadcast_to(f64(gamma)[None, :, None], (B, H, T)).copy()
    ro, rS, _ = oracle.prefill(1, f64(rq), f64(rk), f64(vh), g)
    assert slice_rel_err(f64(o), ro) < TOL[dt] and slice_rel_err(f64(keep), rS) < TOL[dt]
    rn, _ = L.rms_norm(f64(o), f64(wh))
    assert slice_rel_err(f64(out), np.moveaxis(rn, 1, 2).reshape(B, T, C)) < TOL[dt]
    assert out1.shape == (B, 1, C) and torch.isfinite(out1).all()


def test_recurrent_layer_training_step_and_decode(la):
    """Norm -> short convolution -> gated recurrence, its gradients back to the norm's input, and
    the packed prefill and the decode steps of the same layer."""
    B, T, C, dt = 2, 75, 128, torch.bfloat16
    x, res, w = rand(dt, B, T, C, seed=1), rand(dt, B, T, C, seed=2), 1 + 0.2 * rand(torch.float32, C, seed=3)
    gate = torch.sigmoid(rand(torch.float32, B, T, C, seed=4) + 2)
    h0 = rand(torch.float32, B, C, seed=5)
    y, stream = la.rms_norm(x, w, residual=res)
    h, last, kept = la.linear_scan(y, gate, state=h0.clone(), blend=True, checkpoints=True)
    dh, dstream = rand(dt, B, T, C, seed=6), rand(dt, B, T, C, seed=7)
    dy, dgate, d0 = la.linear_scan_backward(y, gate, dh, checkpoints=kept, blend=True, need_dstate0=True)
    dx, dw = la.rms_norm_backward(stream, w, dy, dresidual=dstream)
    # packed: the two rows as two sequences; then token by token from the middle
    cu = torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda")
    ph, plast = la.linear_scan_varlen(y.view(-1, C), gate.view(-1, C), cu, state=h0.clone(), blend=True)
    state = la.linear_scan(y[:, :60].contiguous(), gate[:, :60].contiguous(), state=h0.clone(), blend=True)[1]
    steps = [la.linear_scan_step(y[:, t].contiguous(), gate[:, t].contiguous(), state, blend=True) for t in range(60, T)]
    la.check_status()
    rh, rl, _ = L.linear_scan(f64(y), f64(gate), f64(h0), True)
    for got, ref in ((h, rh), (last, rl), (ph.view(B, T, C), rh), (plast, rl), (torch.stack(steps, 1), rh[:, 60:]), (state, rl)):
        assert slice_rel_err(f64(got), ref, lead=1) < 2.0 ** -7
    (ry, rg, r0), _ = L.linear_scan_backward(f64(y), f64(gate), f64(dh), f64(h0), None, True)
    for got, ref in ((dy, ry), (dgate, rg), (d0, r0)):
        assert slice_rel_err(f64(got), ref, lead=1) < 2.0 ** -7
    (rx, rw), _ = L.rms_norm_backward(f64(stream), f64(w), f64(dy), f64(dstream))
    assert slice_rel_err(f64(dx), rx, lead=1) < 2.0 ** -7 and slice_rel_err(f64(dw)[None], rw[None], lead=1) < 1e-4


def calls(la, seed):
    """Every operator once on fresh inputs: a function and what it returned eagerly."""
    B, T, C, dt = 2, 333, 256, torch.bfloat16
    x, res, dy = (rand(dt, B, T, C, seed=seed + i) for i in range(3))
    gate = torch.sigmoid(rand(torch.float32, B, T, C, seed=seed + 3) + 2)
    w = 1 + 0.2 * rand(torch.float32, C, seed=seed + 4)
    wh = torch.ones(64, device="cuda")
    freqs, _ = la.rotary_frequencies(64)
    cu = torch.tensor([0, 100, 101, B * T], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def run(stream=None):
        h, state, kept = la.linear_scan(x, gate, blend=True, checkpoints=True, stream=stream)
        out = [h, state, *la.linear_scan_backward(x, gate, dy, checkpoints=kept, blend=True, need_dstate0=True,
                                                  stream=stream)]
        out += la.linear_scan_backward(x, gate, dy, blend=True, need_dstate0=True, stream=stream)
        out += la.linear_scan_varlen(x.view(-1, C), gate.view(-1, C), cu, stream=stream)
        q, k = la.rotary(x, dy, freqs=freqs, d=64, stream=stream)
        out += [q, k, la.rotary_backward(q, freqs=freqs, token_major=True, stream=stream)]
        y, s = la.rms_norm(x, w, residual=res, stream=stream)
        q8, sc, _ = la.rms_norm(x, w, residual=res, fp8=True, group=128, stream=stream)
        out += [y, s, q8.view(torch.uint8), sc, *la.rms_norm_backward(s, w, dy, dresidual=res, stream=stream)]
        out += [la.rms_norm_heads(q, wh, stream=stream), *la.rms_norm_heads_backward(q, wh, x, stream=stream)]
        return out

    return run


def test_other_streams(la):
    run = calls(la, 10)
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = run(side)
    with torch.cuda.stream(side):
        also = run()
    side.synchronize()
    for a, b, c in zip(want, got, also):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_two_captured_graphs_replayed_together(la):
    """Two graphs over the same operators, replayed at once on two streams: no shared workspace."""
    runs, graphs, outs = [calls(la, 20), calls(la, 40)], [], []
    want = [[t.clone() for t in r()] for r in runs]
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)
    la.check_status()


def test_two_threads_at_once(la):
    runs = [calls(la, 60), calls(la, 80)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(10):
            got = runs[i](s)
            s.synchronize()
            bad.extend(k for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_launches_are_counted_and_timed(la):
    x, gate = rand(torch.bfloat16, 1, 64, 64), torch.rand(1, 64, 64, device="cuda")
    n = la.kernel_launches()
    la.linear_scan(x, gate)
    assert la.kernel_launches() == n + 1
    la.launch_timing(True)
    try:
        la.rms_norm_backward(x, torch.ones(64, device="cuda"), x)
        times = la.launch_times()
    finally:
        la.launch_timing(False)
    assert len(times) == 2 and all(t > 0 for t in times)


FIRST = """
import torch
import gated_delta_rule_attention_b200 as la
x = torch.randn(2, 100, 256, device="cuda").to(torch.bfloat16)
gate = torch.rand(2, 100, 256, device="cuda")
w, wh = torch.ones(256, device="cuda"), torch.ones(64, device="cuda")
cu = torch.tensor([0, 50, 200], dtype=torch.int32, device="cuda")
freqs, _ = la.rotary_frequencies(64)
def run():
    h, s, kept = la.linear_scan(x, gate, checkpoints=True)
    out = [h, s, *la.linear_scan_backward(x, gate, x, checkpoints=kept, need_dstate0=True)]
    out += la.linear_scan_varlen(x.view(-1, 256), gate.view(-1, 256), cu)
    q = la.rotary(x, freqs=freqs, d=64)
    out += [q, la.rms_norm_heads(q, wh), *la.rms_norm_backward(x, w, x)]
    return out
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):   # the library's first calls in this process
    got = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
la.check_status()
print("same")
"""


def test_first_calls_may_be_captured(tmp_path):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
