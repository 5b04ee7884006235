"""The operators of a selective state space layer: what is timed, and on which sizes.

Three operators, each direction of them a case kind of its own:

  scan_fwd / scan_bwd / scan_step   the selective scan h_t = exp(delta_t A) h_(t-1) + delta_t x_t B_t,
                                    y_t = (C_t . h_t + D x_t) silu(z_t) over prompts, its gradients,
                                    and one token on a kept state;
  conv_fwd / conv_bwd / conv_step   the short causal convolution before it, in the same three forms;
  rms_fwd / rms_bwd / rms_quant     the RMS norm with the residual's addition, its gradients, and the
                                    norm with an e4m3 output and scales.

``own`` false: plain torch operations in 32 bits.  ``own`` true: the framework's entry points.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
ELEM = {BF16: 2, F32: 4}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # An 8192-token prompt through one layer of width 2048 (4096 channels, 16 states each).
        dict(name="scan fwd prompt", op="scan_fwd", B=1, N=8192, E=4096, S=16, G=1, dtype=BF16,
             gate=True, state=False, ragged=False),
        # Three ragged prompts in fp32 with odd sizes, going on from kept states, no gate.
        dict(name="scan fwd odd f32", op="scan_fwd", B=3, N=1001, E=1537, S=11, G=1, dtype=F32,
             gate=False, state=True, ragged=True),
        # A training step's gradients: two sequences of 4096 tokens, 4096 channels.
        dict(name="scan bwd tokens", op="scan_bwd", B=2, N=4096, E=4096, S=16, G=1, dtype=BF16,
             gate=True, state=False, ragged=False),
        # The same in fp32 with two groups of B and C, ragged, with gradients of the states.
        dict(name="scan bwd odd f32", op="scan_bwd", B=2, N=517, E=1002, S=13, G=2, dtype=F32,
             gate=True, state=True, ragged=True),
        # One decode step of one sequence at the 6.7B-scale width (twice 4096 channels): latency.
        dict(name="scan step one", op="scan_step", B=1, N=1, E=8192, S=16, G=1, dtype=BF16,
             gate=True, state=True, ragged=False),
        # The same for 128 sequences: the states' bytes.
        dict(name="scan step many", op="scan_step", B=128, N=1, E=8192, S=16, G=1, dtype=BF16,
             gate=True, state=True, ragged=False),
        # The prompt's and the training step's convolution, four taps.
        dict(name="conv fwd prompt", op="conv_fwd", B=1, N=8192, E=4096, W=4, dtype=BF16,
             state=False, ragged=False),
        dict(name="conv bwd tokens", op="conv_bwd", B=2, N=4096, E=4096, W=4, dtype=BF16,
             state=False, ragged=False),
        # One decode step's convolution for 8 sequences.
        dict(name="conv step", op="conv_step", B=8, N=1, E=8192, W=4, dtype=BF16, state=True,
             ragged=False),
        # The residual's addition and the norm over two 8192-token sequences of the 6.7B-scale width.
        dict(name="rms fwd tokens", op="rms_fwd", n0=2, n1=8192, d=4096, dtype=BF16, residual=True, pad=0),
        # A training step's gradients of it: 8192 tokens.
        dict(name="rms bwd tokens", op="rms_bwd", n0=1, n1=8192, d=4096, dtype=BF16, residual=True, pad=0),
        # The norm of 512 tokens with e4m3 values and a scale for each 128 of them.
        dict(name="rms quant", op="rms_quant", n0=1, n1=512, d=4096, dtype=BF16, residual=True, pad=0,
             group=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd",
                     "conv_bwd", "conv_step", "rms_fwd", "rms_bwd", "rms_quant"])
    dtype = rng.choice([BF16, F32])
    if op.startswith("rms"):
        d = _log_int(rng, 64, 16384)
        d = d // 8 * 8 if rng.random() < 0.6 else d
        n1 = _log_int(rng, 1, min((1 << 26) // d, 32768))
        case = dict(op=op, n0=1, n1=n1, d=d, dtype=dtype, residual=rng.random() < 0.7,
                    pad=rng.choice([0, 0, 0, 8, 3]))
        if op == "rms_quant":
            case["group"] = rng.choice([0, 128])
        return case
    E = _log_int(rng, 16, 8192)
    E = max(E // 16 * 16, 16) if rng.random() < 0.6 else E
    B = _log_int(rng, 1, 16)
    flags = dict(state=rng.random() < 0.5, ragged=rng.random() < 0.4)
    if op.startswith("conv"):
        N = 1 if op == "conv_step" else _log_int(rng, 1, min((1 << 25) // (B * E), 8192))
        if op == "conv_step":
            flags = dict(state=True, ragged=False)
        return dict(op=op, B=B, N=N, E=E, W=rng.choice([2, 3, 4, 4, 4]), dtype=dtype, **flags)
    S = rng.choice([16, 16, 16, 8, 32, 64, rng.randint(1, 64)])
    G = rng.choice([g for g in (1, 1, 1, 2, 4) if E % g == 0])
    if op == "scan_step":
        B = _log_int(rng, 1, min(256, (1 << 24) // (E * S)))
        return dict(op=op, B=B, N=1, E=E, S=S, G=G, dtype=dtype, gate=rng.random() < 0.6, state=True,
                    ragged=False)
    N = _log_int(rng, 1, min((1 << 29) // (B * E * S), 8192))
    return dict(op=op, B=B, N=N, E=E, S=S, G=G, dtype=dtype, gate=rng.random() < 0.6, **flags)


def work(case):
    e, op = ELEM[case["dtype"]], case["op"]
    if op.startswith("rms"):
        rows, d, r = case["n0"] * case["n1"], case["d"], int(case["residual"])
        if op == "rms_bwd":
            # h, dy and what reaches the residual read, dx written; w read, dw written; rstd read
            return dict(bytes=rows * d * e * (3 + r) + d * 8 + rows * 4, flops=rows * d * 9)
        # x and the residual read, their sum and y written; w; rstd written
        io = rows * d * e * (1 + 2 * r) + d * 4
        if op == "rms_quant":
            groups = math.ceil(d / (case["group"] or d))
            return dict(bytes=io + rows * d + rows * groups * 4, flops=rows * d * 7)
        return dict(bytes=io + rows * d * e + rows * 4, flops=rows * d * 5)
    B, N, E = case["B"], case["N"], case["E"]
    n = B * N * E
    if op.startswith("conv"):
        W = case["W"]
        par, st = E * (W + 1) * 4, B * E * (W - 1) * e
        if op == "conv_bwd":
            # x and dy read, dx written; w and b read, dw and db written
            return dict(bytes=3 * n * e + 2 * par + (3 * st if case["state"] else 0),
                        flops=n * (6 * W + 12))
        return dict(bytes=2 * n * e + par + st * (2 if case["state"] else 1), flops=n * (2 * W + 6))
    S, G = case["S"], case["G"]
    gate = int(case["gate"])
    bc, par, st = 2 * B * N * G * S * e, E * (S + 2) * 4, B * E * S * 4
    if op == "scan_bwd":
        # x, dt, dy (and z) read, dx, ddt (and dz) written; B, C and the parameters both ways
        return dict(bytes=n * e * (5 + 2 * gate) + 2 * bc + 2 * par + (3 * st if case["state"] else 0),
                    flops=n * (S * 24 + 40))
    # x, dt (and z) read, y written; B, C; the parameters; the states
    return dict(bytes=n * e * (3 + gate) + bc + par + st * (2 if case["state"] else 1),
                flops=n * (S * 7 + 20))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape, scale=1.0):
    return scale * torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _lengths(case, g):
    """Tokens of each sequence of a padded batch: the first is full, one may be empty."""
    if not case["ragged"]:
        return None
    n = (_rand(g, case["B"]) * (case["N"] + 1)).to(torch.int32).clamp(max=case["N"])
    n[0] = case["N"]
    return n


def _prepare_scan(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    B, N, E, S, G = (case[k] for k in ("B", "N", "E", "S", "G"))
    # step sizes of 0.001 to 0.1 on a logarithmic scale, as such layers are initialised
    step = torch.exp(math.log(1e-3) + (math.log(1e-1) - math.log(1e-3)) * _rand(g, E))
    st = dict(case=dict(case),
              A=-(1.0 + torch.arange(S, device="cuda")) * (0.5 + _rand(g, E, S)),
              D=1.0 + _randn(g, E, scale=0.1),
              dt_bias=step + torch.log(-torch.expm1(-step)))
    one = case["op"] == "scan_step"
    rows = (B,) if one else (B, N)
    st["x"] = torch.nn.functional.silu(_randn(g, *rows, E)).to(dt)
    st["dt"] = _randn(g, *rows, E, scale=0.5).to(dt)
    st["B"] = _randn(g, *rows, G, S).to(dt)
    st["C"] = _randn(g, *rows, G, S).to(dt)
    st["z"] = _randn(g, *rows, E).to(dt) if case["gate"] else None
    st["h_in"] = _randn(g, B, E, S, scale=0.3) if case["state"] else None
    st["lengths"] = _lengths(case, g)
    if one:
        st["h"] = torch.empty(B, E, S, device="cuda")
    st["out"] = torch.empty(*rows, E, dtype=dt, device="cuda")
    if case["op"] == "scan_bwd":
        st["dy"] = _randn(g, B, N, E, scale=0.05).to(dt)
        st["dh_out"] = _randn(g, B, E, S, scale=0.05) if case["state"] else None
    return st


def _prepare_conv(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    B, N, E, W = (case[k] for k in ("B", "N", "E", "W"))
    rows = (B,) if case["op"] == "conv_step" else (B, N)
    st = dict(case=dict(case), w=_randn(g, E, W, scale=0.5), b=_randn(g, E, scale=0.1),
              x=_randn(g, *rows, E).to(dt), out=torch.empty(*rows, E, dtype=dt, device="cuda"))
    st["state_in"] = _randn(g, B, W - 1, E).to(dt) if case["state"] else None
    st["lengths"] = _lengths(case, g)
    if case["op"] == "conv_step":
        st["state"] = torch.empty(B, W - 1, E, dtype=dt, device="cuda")
    if case["op"] == "conv_bwd":
        st["dy"] = _randn(g, B, N, E, scale=0.05).to(dt)
        st["dstate_out"] = _randn(g, B, W - 1, E, scale=0.05).to(dt) if case["state"] else None
    return st


def _prepare_rms(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n0, n1, d = case["n0"], case["n1"], case["d"]

    def rows(scale):
        buf = torch.empty(n0, n1, d + case["pad"], dtype=dt, device="cuda")[..., :d]
        return buf.copy_(_randn(g, n0, n1, d, scale=scale) * (1.0 + _rand(g, d)))

    st = dict(case=dict(case), w=1.0 + _randn(g, d, scale=0.1), x=rows(1.0),
              residual=rows(2.0) if case["residual"] else None)
    if case["op"] == "rms_bwd":
        st["dy"] = rows(0.05)
        st["dh"] = rows(0.05) if case["residual"] else None
        st["rstd"] = torch.rsqrt((st["x"].double() ** 2).mean(-1) + EPS).float()
    return st


def prepare(case, seed):
    kind = case["op"].split("_")[0]
    return dict(scan=_prepare_scan, conv=_prepare_conv, rms=_prepare_rms)[kind](case, seed)


# ------------------------------------------------------------------ plain forms
def _live(st, N):
    """[B, N, 1] truth values: the token is one of its sequence's."""
    lengths = st["lengths"]
    if lengths is None:
        return None
    return (torch.arange(N, device=lengths.device) < lengths[:, None])[..., None]


def _recurrence(a, b):
    """h_t = a_t h_(t-1) + b_t along dimension 1 by doubling."""
    N, k = a.shape[1], 1
    while k < N:
        b = torch.cat([b[:, :k], b[:, k:] + a[:, k:] * b[:, :-k]], 1)
        if 2 * k < N:
            a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _groups(t, E):
    """B or C [.., G, S] for each channel: [.., E, S]."""
    t = t.float()
    return t[..., None, :].expand(*t.shape[:-1], E // t.shape[-2], t.shape[-1]).reshape(
        *t.shape[:-2], E, t.shape[-1])


def _plain_scan_parts(st):
    x, E = st["x"].float(), st["case"]["E"]
    pre = st["dt"].float() + st["dt_bias"]
    delta = _softplus(pre)
    live = _live(st, st["case"]["N"])
    if live is not None:
        delta = torch.where(live, delta, 0.0)
    a = torch.exp(delta[..., None] * st["A"])
    Bm, Cm = _groups(st["B"], E), _groups(st["C"], E)
    b = (delta * x)[..., None] * Bm
    if st["h_in"] is not None:
        b[:, 0] += a[:, 0] * st["h_in"]
    return x, pre, delta, a, Bm, Cm, _recurrence(a, b), live


def _plain_scan_fwd(st):
    x, _, _, _, _, Cm, h, live = _plain_scan_parts(st)
    y = (h * Cm).sum(-1) + st["D"] * x
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    if live is not None:
        y = torch.where(live, y, 0.0)
    return dict(y=y.to(st["x"].dtype), h=h[:, -1].contiguous())


def _plain_scan_step(st):
    x = st["x"].float()
    delta = _softplus(st["dt"].float() + st["dt_bias"])
    Bm, Cm = _groups(st["B"], st["case"]["E"]), _groups(st["C"], st["case"]["E"])
    h = torch.exp(delta[..., None] * st["A"]) * st["h_in"] + (delta * x)[..., None] * Bm
    y = (h * Cm).sum(-1) + st["D"] * x
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    return dict(y=y.to(st["x"].dtype), h=h)


def _plain_scan_bwd(st):
    case, dt = st["case"], st["x"].dtype
    B, N, E, S, G = (case[k] for k in ("B", "N", "E", "S", "G"))
    x, pre, delta, a, Bm, Cm, h, live = _plain_scan_parts(st)
    dy = st["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    out = dict()
    ds = dy
    if st["z"] is not None:
        z = st["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        s = (h * Cm).sum(-1) + st["D"] * x
        out["dz"] = (dy * s * sig * (1.0 + z * (1.0 - sig))).to(dt)
        ds = dy * z * sig
    # g_t = C_t ds_t + a_(t+1) g_(t+1), from the last token to the first
    c = ds[..., None] * Cm
    if st["dh_out"] is not None:
        c[:, -1] += st["dh_out"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _recurrence(later.flip(1), c.flip(1)).flip(1)
    del later, c
    before = torch.cat([(torch.zeros_like(h[:, 0]) if st["h_in"] is None else st["h_in"])[:, None],
                        h[:, :-1]], 1)
    p = a * before  # exp(delta_t A) h_(t-1)
    gp = g * p
    gb = (g * Bm).sum(-1)
    ddelta = x * gb + (gp * st["A"]).sum(-1)
    dx = delta * gb + st["D"] * ds
    ddt = ddelta / (1.0 + torch.exp(-pre))
    if live is not None:
        ddt = torch.where(live, ddt, 0.0)
    out.update(dx=dx.to(dt), ddt=ddt.to(dt), dA=(gp * delta[..., None]).sum((0, 1)),
               dD=(ds * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    out["dB"] = (g * (delta * x)[..., None]).reshape(B, N, G, E // G, S).sum(3).to(dt)
    out["dC"] = (h * ds[..., None]).reshape(B, N, G, E // G, S).sum(3).to(dt)
    if st["h_in"] is not None:
        out["dh_in"] = a[:, 0] * g[:, 0]
    return out


def _plain_conv_parts(st):
    """The inputs with the state before them [B, W-1+N, E], and the sums before silu."""
    case, x = st["case"], st["x"].float()
    B, N, E, W = (case[k] for k in ("B", "N", "E", "W"))
    x = x.reshape(B, N, E)
    first = st["state_in"]
    first = torch.zeros(B, W - 1, E, device=x.device) if first is None else first.float()
    seq = torch.cat([first, x], 1)
    pre = st["b"].expand(B, N, E)
    for k in range(W):
        pre = pre + st["w"][:, k] * seq[:, k:k + N]
    return seq, pre


def _after(st, seq):
    """Indices [B, W-1, E] into seq of the last W-1 inputs of each sequence."""
    case = st["case"]
    last = torch.arange(case["W"] - 1, device=seq.device) + (
        case["N"] if st["lengths"] is None else st["lengths"][:, None].long())
    return last.expand(case["B"], -1)[..., None].expand(-1, -1, case["E"])


def _plain_conv_fwd(st):
    seq, pre = _plain_conv_parts(st)
    y = _silu(pre)
    live = _live(st, st["case"]["N"])
    if live is not None:
        y = torch.where(live, y, 0.0)
    dt = st["x"].dtype
    return dict(y=y.reshape(st["x"].shape).to(dt), state=seq.gather(1, _after(st, seq)).to(dt))


def _plain_conv_bwd(st):
    case, dt = st["case"], st["x"].dtype
    N, W = case["N"], case["W"]
    seq, pre = _plain_conv_parts(st)
    sig = 1.0 / (1.0 + torch.exp(-pre))
    dpre = st["dy"].float() * sig * (1.0 + pre * (1.0 - sig))
    live = _live(st, N)
    if live is not None:
        dpre = torch.where(live, dpre, 0.0)
    dseq = torch.zeros_like(seq)
    dw = torch.empty_like(st["w"])
    for k in range(W):
        dseq[:, k:k + N] += st["w"][:, k] * dpre
        dw[:, k] = (dpre * seq[:, k:k + N]).sum((0, 1))
    if st["dstate_out"] is not None:
        dseq.scatter_add_(1, _after(st, seq), st["dstate_out"].float())
    out = dict(dx=dseq[:, W - 1:].to(dt), dw=dw, db=dpre.sum((0, 1)))
    if st["state_in"] is not None:
        out["dstate_in"] = dseq[:, :W - 1].to(dt)
    return out


def _plain_rms(st):
    """The sum as it is kept (rounded to the inputs' type), its rstd and the normalised row."""
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(h.dtype)
    f = h.float()
    rstd = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    return h, rstd[..., 0], f * rstd * st["w"]


def _plain_rms_fwd(st):
    h, rstd, y = _plain_rms(st)
    out = dict(y=y.to(h.dtype), rstd=rstd)
    if st["residual"] is not None:
        out["h"] = h
    return out


def _blocks(case, t):
    """[.., groups, group] of rows padded with zeros to whole groups."""
    d, size = case["d"], case["group"] or case["d"]
    return torch.nn.functional.pad(t, (0, -d % size)).reshape(*t.shape[:-1], -1, size)


def _values(case, q, scales):
    """What e4m3 values and their groups' scales stand for, in bf16 (as a product takes them up)."""
    values = _blocks(case, q.float()) * scales[..., None]
    return values.flatten(-2)[..., :case["d"]].to(torch.bfloat16)


def _plain_rms_quant(st):
    case = st["case"]
    h, _, _ = _plain_rms(st)
    f = h.double()  # (a value next to the border between two e4m3 values)
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * st["w"]
    blocks = _blocks(case, y)
    scales = blocks.abs().amax(-1) / 448.0
    safe = torch.where(scales > 0, scales, 1.0)
    q = (blocks / safe[..., None]).clamp(-448.0, 448.0).float().to(torch.float8_e4m3fn)
    scales = scales.float()
    out = dict(y=_values(case, q.flatten(-2)[..., :case["d"]], scales), scales=scales)
    if st["residual"] is not None:
        out["h"] = h
    return out


def _plain_rms_bwd(st):
    h, dy, r = st["x"].float(), st["dy"].float(), st["rstd"][..., None]
    n, g = h * r, dy * st["w"]
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return dict(dx=dx.to(st["x"].dtype), dw=(dy * n).sum((0, 1)))


_PLAIN = dict(scan_fwd=_plain_scan_fwd, scan_bwd=_plain_scan_bwd, scan_step=_plain_scan_step,
              conv_fwd=_plain_conv_fwd, conv_bwd=_plain_conv_bwd, conv_step=_plain_conv_fwd,
              rms_fwd=_plain_rms_fwd, rms_bwd=_plain_rms_bwd, rms_quant=_plain_rms_quant)


# ------------------------------------------------------------------ one pass
def _run_own(st):
    from linear_recurrent_sequence_gb300 import retention as R
    case = st["case"]
    op = case["op"]
    if op.startswith("scan"):
        args = [st[k] for k in ("x", "dt", "A", "B", "C")]
        kw = dict(D=st["D"], z=st["z"], dt_bias=st["dt_bias"])
        if op == "scan_step":
            # (without h_out the step updates the state in place)
            y = R.selective_scan_step(*args, st["h_in"], h_out=st["h"], out=st["out"], **kw)
            return dict(y=y, h=st["h"])
        kw.update(h_in=st["h_in"], lengths=st["lengths"])
        if op == "scan_fwd":
            y, h = R.selective_scan_fwd(*args, out=st["out"], **kw)
            return dict(y=y, h=h)
        grads = R.selective_scan_bwd(*args, st["dy"], dh_out=st["dh_out"], **kw)
        return {k: v for k, v in grads._asdict().items() if v is not None}
    if op == "conv_step":
        y = R.causal_conv_step(st["x"], st["w"], st["b"], st["state_in"], state_out=st["state"],
                               out=st["out"])
        return dict(y=y, state=st["state"])
    if op == "conv_fwd":
        y, state = R.causal_conv_fwd(st["x"], st["w"], st["b"], state_in=st["state_in"],
                                     lengths=st["lengths"], out=st["out"])
        return dict(y=y, state=state)
    if op == "conv_bwd":
        dx, dw, db, ds = R.causal_conv_bwd(st["x"], st["w"], st["b"], st["dy"],
                                           state_in=st["state_in"], dstate_out=st["dstate_out"],
                                           lengths=st["lengths"])
        out = dict(dx=dx, dw=dw, db=db)
        if ds is not None:
            out["dstate_in"] = ds
        return out
    if op == "rms_bwd":
        dx, dw = R.rmsnorm_bwd(st["x"], st["dy"], st["w"], st["rstd"], dh=st["dh"])
        return dict(dx=dx, dw=dw)
    if op == "rms_quant":
        q, scales, h = R.rmsnorm_quant(st["x"], st["w"], residual=st["residual"], eps=EPS,
                                       group=case["group"])
        out = dict(y=_values(case, q, scales), scales=scales)
    else:
        y, h, rstd = R.rmsnorm_fwd(st["x"], st["w"], residual=st["residual"], eps=EPS)
        out = dict(y=y, rstd=rstd)
    if st["residual"] is not None:
        out["h"] = h
    return out


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_scan(st):
    """The recurrence token by token, and its gradients by the chain rule from the last one."""
    case = st["case"]
    B, N, E, S, G = (case[k] for k in ("B", "N", "E", "S", "G"))
    A, D, bias = st["A"].double(), st["D"].double(), st["dt_bias"].double()

    def per_token(t, *shape):
        return t.double().reshape(B, N, *shape)

    x, u = per_token(st["x"], E), per_token(st["dt"], E) + bias
    Bs, Cs = per_token(st["B"], G, 1, S), per_token(st["C"], G, 1, S)
    delta = torch.logaddexp(u, torch.zeros_like(u))
    n = torch.full((B,), N, device=x.device) if st["lengths"] is None else st["lengths"].long()
    there = torch.arange(N, device=x.device)[None] < n[:, None]
    back = case["op"] == "scan_bwd"
    h = torch.zeros(B, E, S, dtype=torch.float64, device=x.device) if st["h_in"] is None else st["h_in"].double()
    first, kept, s = h, [], torch.empty(B, N, E, dtype=torch.float64, device=x.device)
    wide = (B, G, E // G, S)
    for t in range(N):
        new = torch.exp(delta[:, t, :, None] * A) * h
        new = new + ((delta[:, t] * x[:, t]).reshape(B, G, -1, 1) * Bs[:, t]).reshape(B, E, S)
        h = torch.where(there[:, t, None, None], new, h)
        s[:, t] = (h.reshape(wide) * Cs[:, t]).sum(-1).reshape(B, E) + D * x[:, t]
        if back:
            kept.append(h)
    z = None if st["z"] is None else per_token(st["z"], E)
    gate = 1.0 if z is None else z * torch.sigmoid(z)
    if not back:
        y = s * gate * there[..., None]
        return dict(y=y.reshape(st["x"].shape), h=h)
    dy = per_token(st["dy"], E) * there[..., None]
    ds = dy * gate
    out = dict()
    if z is not None:
        sg = torch.sigmoid(z)
        out["dz"] = dy * s * (sg + z * sg * (1.0 - sg))
    g = torch.zeros_like(h) if st["dh_out"] is None else st["dh_out"].double()
    out.update({k: torch.zeros(B, N, E, dtype=torch.float64, device=x.device) for k in ("dx", "ddt")})
    out["dA"] = torch.zeros_like(A)
    out.update({k: torch.zeros(B, N, G, S, dtype=torch.float64, device=x.device) for k in ("dB", "dC")})
    for t in range(N - 1, -1, -1):
        m = there[:, t, None]
        g = g + (ds[:, t].reshape(B, G, -1, 1) * Cs[:, t]).reshape(B, E, S)
        out["dC"][:, t] = (kept[t].reshape(wide) * ds[:, t].reshape(B, G, -1, 1)).sum(2)
        out["dB"][:, t] = (g.reshape(wide) * (delta[:, t] * x[:, t] * m).reshape(B, G, -1, 1)).sum(2)
        into = (g.reshape(wide) * Bs[:, t]).sum(-1).reshape(B, E)
        decay = torch.exp(delta[:, t, :, None] * A)
        through = g * decay * (kept[t - 1] if t else first) * m[..., None]
        out["dx"][:, t] = (into * delta[:, t] + ds[:, t] * D) * m
        out["ddt"][:, t] = (into * x[:, t] * m + (through * A).sum(-1)) * torch.sigmoid(u[:, t])
        out["dA"] += (through * delta[:, t, :, None]).sum(0)
        g = torch.where(m[..., None], g * decay, g)
    out["dD"] = (ds * x).sum((0, 1))
    out["ddt_bias"] = out["ddt"].sum((0, 1))
    if st["h_in"] is not None:
        out["dh_in"] = g
    return out


def _exact_conv(st):
    """Tap by tap with explicit positions before the first token."""
    case = st["case"]
    B, N, E, W = (case[k] for k in ("B", "N", "E", "W"))
    x = st["x"].double().reshape(B, N, E)
    w = st["w"].double()
    lag = W - 1
    old = None if st["state_in"] is None else st["state_in"].double()
    n = [N] * B if st["lengths"] is None else [int(v) for v in st["lengths"].tolist()]

    def shifted(i):  # the inputs i tokens earlier
        head = x.new_zeros(B, min(i, N), E)
        if old is not None and i:
            head = old[:, lag - i:][:, :min(i, N)]
        return torch.cat([head, x[:, :max(N - i, 0)]], 1)

    pre = st["b"].double() + sum(w[:, lag - i] * shifted(i) for i in range(W))
    sg = torch.sigmoid(pre)
    if case["op"] != "conv_bwd":
        y = pre * sg
        state = x.new_zeros(B, lag, E)
        for i in range(B):
            y[i, n[i]:] = 0.0
            for k in range(lag):
                at = n[i] - lag + k
                if at >= 0:
                    state[i, k] = x[i, at]
                elif old is not None:
                    state[i, k] = old[i, lag + at]
        return dict(y=y.reshape(st["x"].shape), state=state)
    d = st["dy"].double() * (sg + pre * sg * (1.0 - sg))
    for i in range(B):
        d[i, n[i]:] = 0.0
    dx, dold = torch.zeros_like(x), x.new_zeros(B, lag, E)
    for i in range(W):
        back = d * w[:, lag - i]
        dx[:, :max(N - i, 0)] += back[:, i:]
        for t in range(min(i, N)):
            dold[:, lag - i + t] += back[:, t]
    if st["dstate_out"] is not None:
        for i in range(B):
            for k in range(lag):
                at = n[i] - lag + k
                (dx[i] if at >= 0 else dold[i])[at if at >= 0 else lag + at] += st["dstate_out"][i, k].double()
    out = dict(dx=dx, dw=torch.stack([(d * shifted(lag - k)).sum((0, 1)) for k in range(W)], 1),
               db=d.sum((0, 1)))
    if old is not None:
        out["dstate_in"] = dold
    return out


def _exact_rms(st):
    case, dt = st["case"], st["x"].dtype
    w = st["w"].double()
    if case["op"] == "rms_bwd":
        h, dy, r = st["x"].double(), st["dy"].double(), st["rstd"].double()
        inner = (dy * w * h).sum(-1) * r ** 3 / case["d"]
        dx = dy * w * r[..., None] - h * inner[..., None]
        if st["dh"] is not None:
            dx = dx + st["dh"].double()
        return dict(dx=dx, dw=(dy * h * r[..., None]).sum((0, 1)))
    # the sum is kept in the inputs' type, and what is kept is normalised
    h = st["x"] if st["residual"] is None else (st["x"].double() + st["residual"].double()).to(dt)
    f = h.double()
    rstd = 1.0 / torch.sqrt((f * f).sum(-1) / case["d"] + EPS)
    y = f * rstd[..., None] * w
    if case["op"] == "rms_fwd":
        out = dict(y=y, rstd=rstd)
    else:
        size = case["group"] or case["d"]
        scales = torch.stack([c.abs().amax(-1) for c in y.split(size, -1)], -1) / 448.0
        q = torch.cat([(c / s[..., None]) for c, s in zip(y.split(size, -1), scales.unbind(-1))], -1)
        q = torch.nan_to_num(q).float().to(torch.float8_e4m3fn).double()
        parts = [c * s[..., None] for c, s in zip(q.split(size, -1), scales.unbind(-1))]
        out = dict(y=torch.cat(parts, -1), scales=scales)
    if st["residual"] is not None:
        out["h"] = h.double()
    return out


def exact(case, seed):
    """The definitions in 64 bits, apart from the plain forms."""
    kind = case["op"].split("_")[0]
    return dict(scan=_exact_scan, conv=_exact_conv, rms=_exact_rms)[kind](prepare(case, seed))
