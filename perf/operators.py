"""What the layer operators around the linear-attention kernels are measured on.

Three operators: the gated linear recurrence with a vector state (``linear_scan``), rotary
positions of q and k (``rotary``), and the root-mean-square norm with the residual's addition
and an optional 8-bit output (``rms_norm``).  ``run`` computes a case in plain torch operations
when ``own`` is false and by the package's entry points when it is true; ``exact`` gives the
definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
FP8_MAX = 448.0


def listed():
    return [
        # A recurrent layer's prefill at the attention benchmark's length and width (16 heads of
        # 128): the largest case, bandwidth alone.
        dict(name="scan_prefill", kind="scan", dtype="bf16", B=2, T=32768, C=2048, blend=False),
        # A training step of such a layer: the forward call that keeps its checkpoints, and the
        # backward call.
        dict(name="scan_train", kind="scan_grad", dtype="bf16", B=4, T=4096, C=2048, blend=True),
        # One long sequence of a narrow fp32 layer, odd length: little parallelism in channels.
        dict(name="scan_narrow", kind="scan", dtype="fp32", B=1, T=50001, C=192, blend=True),
        # A serving step's prompts, packed, each resumed from its own cached state.
        dict(name="scan_packed", kind="scan_packed", dtype="bf16", N=61, T=20011, C=1024, blend=False),
        # One token for 256 sequences (the decode benchmark's batch, 32 heads of 128).
        dict(name="scan_step", kind="scan_step", dtype="bf16", N=256, C=4096, blend=True),
        # q and k of a constant-decay layer's prefill, from the projections to head-major rows.
        dict(name="rotary_prefill", kind="rotary", dtype="bf16", B=8, T=8192, H=16, Hk=16, d=128, r=128,
             interleaved=False, start=0, base=10000.0, factor=1.0, scale=1.0),
        # The gradient of a layer that rotates a quarter of each head, shared key heads, far positions
        # of a context stretched eightfold, odd length, fp32.
        dict(name="rotary_grad", kind="rotary_grad", dtype="fp32", B=1, T=9001, H=32, Hk=8, d=128, r=32,
             interleaved=True, start=1000000, base=500000.0, factor=8.0, scale=1.2),
        # One token for 256 sequences, each at its own position.
        dict(name="rotary_step", kind="rotary_step", dtype="bf16", N=256, H=32, Hk=8, d=128, r=64,
             interleaved=False, start=262144, base=1000000.0, factor=4.0, scale=1.1),
        # A training step of the pre-norm in front of a layer's projections: forward and backward.
        dict(name="norm_train", kind="norm_grad", dtype="bf16", R=16384, C=2048),
        # The pre-norm of a prefill whose projections take e4m3 with a scale for each 128 columns.
        dict(name="norm_fp8", kind="norm", dtype="bf16", R=32768, C=4096, residual=True, group=128),
        # The norm after the attention, head-major in and token-major out.
        dict(name="norm_heads", kind="norm_heads", dtype="bf16", B=4, H=16, T=4096, d=128),
        # The pre-norm of a decode step, e4m3 with one scale a row.
        dict(name="norm_step", kind="norm", dtype="bf16", R=256, C=4096, residual=True, group=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the listed ones' ranges (a call moves at most about 0.5 GB)."""
    kind = rng.choice(["scan", "scan", "scan_grad", "scan_packed", "scan_step", "rotary", "rotary_grad",
                       "rotary_step", "norm", "norm", "norm_grad", "norm_heads"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    most = 1 << 25   # elements of the largest tensor
    if kind in ("scan", "scan_grad", "scan_packed"):
        C = _log(rng, 48, 4096)
        if rng.random() < 0.7:
            C = max(8, C // 8 * 8)
        T = _log(rng, 16, min(60000, most // C))
        c = dict(kind=kind, dtype=dtype, T=T, C=C, blend=rng.random() < 0.5)
        if kind == "scan_packed":
            c["N"] = min(T, _log(rng, 1, 200))
        else:
            c["B"] = rng.randint(1, max(1, min(4, most // (C * T))))
        return c
    if kind == "scan_step":
        return dict(kind=kind, dtype=dtype, N=_log(rng, 1, 512), C=_log(rng, 48, 8192), blend=rng.random() < 0.5)
    if kind.startswith("rotary"):
        d = rng.choice([64, 128])
        H = rng.choice([1, 2, 5, 8, 16, 32])
        Hk = rng.choice([h for h in (1, 2, 4, 5, 8, 16, 32) if H % h == 0])
        c = dict(kind=kind, dtype=dtype, H=H, Hk=Hk, d=d, r=rng.choice([d, d // 2, d // 4, 24]),
                 interleaved=rng.random() < 0.5, start=_log(rng, 1, 2000000) - 1,
                 base=rng.choice([10000.0, 500000.0]), factor=rng.choice([1.0, 4.0, 16.0]),
                 scale=rng.choice([1.0, 1.1]))
        if kind == "rotary_step":
            c["N"] = _log(rng, 1, 512)
        else:
            c["T"] = _log(rng, 16, min(40000, most // (H * d)))
            c["B"] = rng.randint(1, max(1, min(4, most // (H * d * c["T"]))))
        return c
    if kind == "norm_heads":
        H, d = rng.choice([1, 4, 6, 16, 32]), rng.choice([64, 128])
        return dict(kind=kind, dtype=dtype, B=rng.randint(1, 4), H=H, d=d, T=_log(rng, 1, most // (4 * H * d)))
    C = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        C = C // 8 * 8
    group = rng.choice([-1, 0, 128]) if kind == "norm" else -1   # -1: no 8-bit output
    if group == 128:
        C = max(128, C // 128 * 128)
    c = dict(kind=kind, dtype=dtype, R=_log(rng, 1, min(60000, most // C)), C=C)
    if kind == "norm":
        c |= dict(residual=rng.random() < 0.7, group=group)
    return c


# ------------------------------------------------------------------------------- inputs

def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _gates(g, *shape):
    """Decays in (0, 1): exp(-softplus(r) rate), with one rate a channel, from memories of a few
    tokens to memories of thousands."""
    rate = torch.exp(torch.rand(shape[-1], generator=g, device="cuda") * math.log(1000.0)) / 1000.0
    return torch.exp(-torch.nn.functional.softplus(_rand(g, *shape)).mul_(rate))


def _lengths(case, seed):
    """Lengths of the packed sequences, ragged, some of them 1 and one of them 0 (from the seed)."""
    g = torch.Generator().manual_seed(seed)
    N, T = case["N"], case["T"]
    if N == 1:
        return [T]
    w = torch.exp(torch.randn(N, generator=g) * 1.0)
    w[torch.randint(N, (1,), generator=g)] = 0
    n = torch.floor(w / w.sum() * (T - N)).long() + (w > 0).long()
    n[int(torch.argmax(n))] += T - int(n.sum())
    return n.tolist()


def frequencies(case):
    """Angles per position in 64 bits, positions divided by the stretch of the context."""
    j = torch.arange(case["r"] // 2, dtype=torch.float64, device="cuda")
    return case["base"] ** (-2.0 * j / case["r"]) / case["factor"]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, kind, s = DTYPES[case["dtype"]], case["kind"], {"case": case}
    if kind in ("scan", "scan_grad"):
        shape = (case["B"], case["T"], case["C"])
        s |= dict(x=_rand(g, *shape).to(dt), gate=_gates(g, *shape))
        if kind == "scan_grad":
            s |= dict(dh=_rand(g, *shape).to(dt), state0=_rand(g, case["B"], case["C"]),
                      dstate=_rand(g, case["B"], case["C"]))
    elif kind == "scan_packed":
        shape = (case["T"], case["C"])
        n = torch.tensor([0] + _lengths(case, seed))
        s |= dict(x=_rand(g, *shape).to(dt), gate=_gates(g, *shape), state=_rand(g, case["N"], case["C"]),
                  cu=n.cumsum(0).to(torch.int32).cuda())
    elif kind == "scan_step":
        shape = (case["N"], case["C"])
        s |= dict(x=_rand(g, *shape).to(dt), gate=_gates(g, *shape), state=_rand(g, *shape))
    elif kind in ("rotary", "rotary_grad", "rotary_step"):
        H, Hk, d = case["H"], case["Hk"], case["d"]
        s["freqs"] = frequencies(case)
        if kind == "rotary":
            shapes = (case["B"], case["T"], H * d), (case["B"], case["T"], Hk * d)
        elif kind == "rotary_grad":
            shapes = (case["B"], H, case["T"], d), (case["B"], Hk, case["T"], d)
        else:
            shapes = (case["N"], H * d), (case["N"], Hk * d)
            s["positions"] = torch.randint(case["start"] + 1, (case["N"],), generator=g, device="cuda",
                                           dtype=torch.int32)
        s |= dict(q=_rand(g, *shapes[0]).to(dt), k=_rand(g, *shapes[1]).to(dt))
    elif kind in ("norm", "norm_grad"):
        shape = (case["R"], case["C"])
        s |= dict(x=_rand(g, *shape).to(dt), w=1 + 0.2 * _rand(g, case["C"]))
        if kind == "norm_grad" or case["residual"]:
            s["residual"] = (2 * _rand(g, *shape)).to(dt)
        if kind == "norm_grad":
            s |= dict(dy=_rand(g, *shape).to(dt), dres=_rand(g, *shape).to(dt))
    else:
        s |= dict(x=(0.3 * _rand(g, case["B"], case["H"], case["T"], case["d"])).to(dt),
                  w=1 + 0.2 * _rand(g, case["d"]))
    return s


# ------------------------------------------------------------------------------- plain forms

def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim -2 from zero, by doubling the span of (a, b) pairs."""
    a, b, k, T = a.clone(), b.clone(), 1, a.shape[-2]
    while k < T:
        b[..., k:, :] += a[..., k:, :] * b[..., :-k, :].clone()
        a[..., k:, :] *= a[..., :-k, :].clone()
        k *= 2
    return b


def _from(a, b, first):
    """b with the state before the first row taken in."""
    b = b.clone()
    b[..., 0, :] += a[..., 0, :] * first
    return b


def _inputs(case, x, a):
    x = x.float()
    return (1 - a) * x if case["blend"] else x


def _plain_scan(s):
    case, a = s["case"], s["gate"]
    h = _scan(a, _inputs(case, s["x"], a))
    return h.to(s["x"].dtype), h[..., -1, :].clone()


def _plain_scan_grad(s):
    case, a, x = s["case"], s["gate"], s["x"]
    h = _scan(a, _from(a, _inputs(case, x, a), s["state0"]))
    before = torch.cat([s["state0"].unsqueeze(-2), h[..., :-1, :]], -2)
    dh = s["dh"].float()
    dh[..., -1, :] += s["dstate"]
    later = torch.cat([a[..., 1:, :], torch.zeros_like(a[..., :1, :])], -2)
    lam = _scan(later.flip(-2), dh.flip(-2)).flip(-2)
    if case["blend"]:
        dx, da = (1 - a) * lam, lam * (before - x.float())
    else:
        dx, da = lam, lam * before
    return h.to(x.dtype), h[..., -1, :].clone(), dx.to(x.dtype), da, a[..., 0, :] * lam[..., 0, :]


def _plain_packed(s):
    case, cu, state = s["case"], s["cu"].long(), s["state"]
    a, b = s["gate"].clone(), _inputs(case, s["x"], s["gate"]).clone()
    held = cu[1:] > cu[:-1]
    first, last = cu[:-1][held], cu[1:][held] - 1
    b[first] += a[first] * state[held]
    a[first] = 0
    h = _scan(a, b)
    state[held] = h[last]
    return h.to(s["x"].dtype), state


def _plain_step(s):
    a = s["gate"]
    s["state"].mul_(a).add_(_inputs(s["case"], s["x"], a))
    return s["state"].to(s["x"].dtype), s["state"]


def _rotate(case, x, pos, freqs, sign):
    """x [..., T, H, d] at pos [..., T]: the first r values of each head in pairs, the rest as they are."""
    r = case["r"]
    angle = (pos.double().unsqueeze(-1) * freqs).unsqueeze(-2)
    c, n = case["scale"] * angle.cos().float(), sign * case["scale"] * angle.sin().float()
    y = x.float().clone()
    u, v = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    nu, nv = u * c - v * n, u * n + v * c
    u.copy_(nu)
    v.copy_(nv)
    return y.to(x.dtype)


def _plain_rotary(s):
    case, freqs, d = s["case"], s["freqs"], s["case"]["d"]
    if case["kind"] == "rotary_step":
        pos = s["positions"]
        return [_rotate(case, x.unflatten(-1, (-1, d)), pos, freqs, 1) for x in (s["q"], s["k"])]
    pos = (case["start"] + torch.arange(case["T"], device="cuda")).expand(case["B"], -1)
    if case["kind"] == "rotary":
        return [_rotate(case, x.unflatten(-1, (-1, d)), pos, freqs, 1).transpose(1, 2).contiguous()
                for x in (s["q"], s["k"])]
    return [_rotate(case, x.transpose(1, 2), pos, freqs, -1).flatten(2) for x in (s["q"], s["k"])]


def _eight(y, group):
    """e4m3 values and the scales of rows (group 0) or of `group` columns: the largest is 448."""
    u = y.unflatten(-1, (-1, group or y.shape[-1]))
    top = u.abs().amax(-1)
    scale = torch.where(top > 0, (top / FP8_MAX).clamp(min=torch.finfo(torch.float32).tiny), 1.0)
    q = (u / scale.unsqueeze(-1)).clamp(-FP8_MAX, FP8_MAX).flatten(-2).to(torch.float8_e4m3fn)
    return q, scale


def _plain_norm(s):
    case, x, w = s["case"], s["x"], s["w"]
    if case["kind"] == "norm_heads":
        x = x.transpose(1, 2)
    h = (x.float() + s["residual"].float()).to(x.dtype) if "residual" in s else x
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
    y = f * rstd * w
    if case["kind"] == "norm_heads":
        return y.flatten(2).to(x.dtype)
    out = [h] if "residual" in s else []
    if case["kind"] == "norm_grad":
        dy = s["dy"].float()
        n = f * rstd
        t = dy * w
        dx = rstd * (t - n * (t * n).mean(-1, keepdim=True)) + s["dres"].float()
        return [y.to(x.dtype)] + out + [dx.to(x.dtype), (dy * n).sum(0)]
    return out + (list(_eight(y, case["group"])) if case["group"] >= 0 else [y.to(x.dtype)])


# ------------------------------------------------------------------------------- the package's calls

def _own(s):
    import gated_delta_rule_attention_b200 as la
    case = s["case"]
    kind = case["kind"]
    if kind == "scan":
        return la.linear_scan(s["x"], s["gate"], blend=case["blend"])
    if kind == "scan_grad":
        h, state, kept = la.linear_scan(s["x"], s["gate"], state=s["state0"].clone(), blend=case["blend"],
                                        checkpoints=True)
        dx, dgate, dstate0 = la.linear_scan_backward(s["x"], s["gate"], s["dh"], checkpoints=kept,
                                                     dstate=s["dstate"], blend=case["blend"],
                                                     need_dstate0=True)
        return h, state, dx, dgate, dstate0
    if kind == "scan_packed":
        return la.linear_scan_varlen(s["x"], s["gate"], s["cu"], state=s["state"], blend=case["blend"])
    if kind == "scan_step":
        return la.linear_scan_step(s["x"], s["gate"], s["state"], blend=case["blend"]), s["state"]
    if kind.startswith("rotary"):
        more = dict(interleaved=case["interleaved"], scale=case["scale"])
        if kind == "rotary_step":
            return la.rotary_step(s["q"], s["k"], freqs=s["freqs"], positions=s["positions"], d=case["d"], **more)
        if kind == "rotary":
            return la.rotary(s["q"], s["k"], freqs=s["freqs"], start=case["start"], d=case["d"], **more)
        return la.rotary_backward(s["q"], s["k"], freqs=s["freqs"], start=case["start"], token_major=True, **more)
    if kind == "norm_heads":
        return la.rms_norm_heads(s["x"], s["w"])
    if kind == "norm_grad":
        y, h = la.rms_norm(s["x"], s["w"], residual=s["residual"])
        return (y, h) + la.rms_norm_backward(h, s["w"], s["dy"], dresidual=s["dres"])
    fp8 = case["group"] >= 0
    out = la.rms_norm(s["x"], s["w"], residual=s.get("residual"), fp8=fp8, group=max(case["group"], 0))
    out = out if isinstance(out, tuple) else (out,)
    if "residual" in s:   # (y, h) or (q, scales, h), in the plain form's order
        return [out[-1]] + list(out[:-1])
    return list(out)


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "scan":
        return _plain_scan(state)
    if kind == "scan_grad":
        return _plain_scan_grad(state)
    if kind == "scan_packed":
        return _plain_packed(state)
    if kind == "scan_step":
        return _plain_step(state)
    return _plain_rotary(state) if kind.startswith("rotary") else _plain_norm(state)


def work(case):
    """Every call's inputs read once and outputs written once (a training step is two calls with
    the loss between them: its backward call reads x and the gates again, and a checkpoint row for
    every 32)."""
    e, kind = SIZE[case["dtype"]], case["kind"]
    if kind == "scan":
        n = case["B"] * case["T"] * case["C"]
        return {"bytes": n * (4 + 2 * e) + 4 * case["B"] * case["C"], "flops": 2 * n}
    if kind == "scan_grad":
        n, c = case["B"] * case["T"] * case["C"], case["B"] * case["C"]
        return {"bytes": n * (4 + 2 * e) + n * (8 + 3 * e) + 2 * n // 8 + 16 * c, "flops": 9 * n}
    if kind == "scan_packed":
        n = case["T"] * case["C"]
        return {"bytes": n * (4 + 2 * e) + 8 * case["N"] * case["C"], "flops": 2 * n}
    if kind == "scan_step":
        return {"bytes": case["N"] * case["C"] * (12 + 2 * e), "flops": 2 * case["N"] * case["C"]}
    if kind.startswith("rotary"):
        rows = case["N"] if kind == "rotary_step" else case["B"] * case["T"]
        n = rows * (case["H"] + case["Hk"]) * case["d"]
        return {"bytes": 2 * n * e, "flops": 3 * n * case["r"] / case["d"]}
    if kind == "norm_heads":
        n = case["B"] * case["T"] * case["H"] * case["d"]
        return {"bytes": 2 * n * e, "flops": 4 * n}
    n = case["R"] * case["C"]
    if kind == "norm_grad":
        return {"bytes": 4 * n * e + 4 * n * e + 12 * case["C"], "flops": 14 * n}
    out = e if case["group"] < 0 else 1 + 4 / (case["group"] or case["C"])
    return {"bytes": n * (e * (3 if case["residual"] else 1) + out) + 4 * case["C"], "flops": 5 * n}


# ------------------------------------------------------------------------------- 64 bits

def _walk(a, b, h, resets=None):
    """The recurrence token by token: every h_t, in 64 bits.  a, b [B, T, C]; h [B, C]; resets: the
    state that replaces h in front of a row."""
    out = torch.empty_like(b)
    for t in range(b.shape[1]):
        if resets and t in resets:
            h = resets[t]
        h = torch.addcmul(b[:, t], a[:, t], h, out=out[:, t])
    return out


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    D = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if kind.startswith("scan"):
        a = D["gate"]
        b = D["x"] * (1 - a) if case["blend"] else D["x"]
    if kind == "scan":
        h = _walk(a, b, torch.zeros_like(b[:, 0]))
        return h, h[:, -1]
    if kind == "scan_grad":
        h = _walk(a, b, D["state0"])
        lam, carry = D["dh"].clone(), D["dstate"]
        for t in range(case["T"] - 1, -1, -1):
            lam[:, t] += carry
            carry = a[:, t] * lam[:, t]
        prev = torch.cat([D["state0"][:, None], h[:, :-1]], 1)
        dx = lam * (1 - a) if case["blend"] else lam
        return h, h[:, -1], dx, lam * (prev - D["x"] if case["blend"] else prev), carry
    if kind == "scan_packed":
        cu, state = s["cu"].tolist(), D["state"]
        held = [n for n in range(case["N"]) if cu[n + 1] > cu[n]]
        h = _walk(a[None], b[None], torch.zeros_like(b[:1]), {cu[n]: state[n:n + 1] for n in held})[0]
        for n in held:
            state[n] = h[cu[n + 1] - 1]
        return h, state
    if kind == "scan_step":
        h = a * D["state"] + b
        return h, h
    if kind.startswith("rotary"):
        if kind == "rotary_step":
            pos = s["positions"].double()
        else:
            pos = torch.arange(case["start"], case["start"] + case["T"], device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.full((), case["scale"], dtype=torch.float64, device="cuda").expand(
            pos.shape[0], case["r"] // 2), torch.outer(pos, s["freqs"]))
        out = []
        for x in (D["q"], D["k"]):
            # rows [.., token, head, d] as complex pairs
            x = x.view(*x.shape[:-1], -1, case["d"]) if kind != "rotary_grad" else x.transpose(1, 2)
            part, rest = x[..., :case["r"]], x[..., case["r"]:]
            if case["interleaved"]:
                z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous())
            else:
                z = torch.complex(*part.chunk(2, -1))
            z = z * (turn.conj() if kind == "rotary_grad" else turn)[:, None, :]
            part = torch.stack([z.real, z.imag], -1 if case["interleaved"] else -2).flatten(-2)
            y = torch.cat([part, rest], -1)
            out.append(y.transpose(1, 2).contiguous() if kind == "rotary" else y.flatten(2) if kind == "rotary_grad"
                       else y)
        return out
    # the norms: the stream is stored rounded, by the operator's definition
    h = (D["x"] + D["residual"]).to(s["x"].dtype).double() if "residual" in D else D["x"]
    norm = torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + 1e-6)
    y = h / norm * D["w"]
    if kind == "norm_heads":
        return y.permute(0, 2, 1, 3).reshape(case["B"], case["T"], -1)
    if kind == "norm_grad":
        p = D["dy"] * D["w"]
        dx = p / norm - h * (p * h).sum(-1, keepdim=True) / (h.shape[-1] * norm ** 3) + D["dres"]
        return [y, h, dx, (D["dy"] * h / norm).sum(0)]
    out = [h] if "residual" in D else []
    if case["group"] < 0:
        return out + [y]
    parts = y.view(case["R"], -1, case["group"] or case["C"])
    scale = parts.abs().max(-1).values / FP8_MAX
    return out + [(parts / scale[..., None]).reshape(case["R"], -1), scale]
