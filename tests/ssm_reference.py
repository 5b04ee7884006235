"""64-bit references of the selective scan, the causal convolution and the RMS
norm, token by token, with the error that fp32 arithmetic may make of them.

Errors of the scan, u = 2^-24.  A decay e^(delta A) is 2^(delta A log2(e)) by the
hardware's exponential (2^-22 of itself) of a product whose factors are off by
E_DELTA = 16 u (the step size: exponential, reciprocal and series) and 2 u (A
log2(e) and the product), so it is off by RHO + |delta A| sigma with RHO = 2^-22.
Where decays of many tokens are joined through the sum of their step sizes,
that sum's own error, a chain of at most N / 4 + 64 additions, belongs to sigma.
The error of the state then follows the recurrence
  err_t = a_t err_(t-1) + a_t |h|_(t-1) (RHO + |delta A| sigma) + |u B| tau + 2 u |h|_t
with |h|_t = a_t |h|_(t-1) + |u B| and tau = E_DELTA + 3 u, and that of the
gradient's recurrence the same one backwards (tau = 32 u: ds carries silu's
error, below 16 u).  What a result adds up from them is off by the largest
relative error R of the two for each factor, and u for each addition.
"""
import torch

U = 2.0 ** -24
RHO, E_DELTA = 2.0 ** -22, 16 * U


def half_ulp(ref, dtype):
    """Half a step of the result's type (fp32: included in the other bounds)."""
    if dtype == torch.bfloat16:
        return ref.abs() * 2.0 ** -8 + 1e-38
    return ref.abs() * U


def expand(t, E):
    """B or C [.., G, S] for each channel [.., E, S]."""
    return t.double().repeat_interleave(E // t.shape[-2], dim=-2)


def scan(x, dt, A, B, C, D=None, z=None, bias=None, softplus=True, h_in=None, lengths=None, dy=None, dh_out=None):
    """Results and error bounds: {name: (value, bound)} of y, h and with dy of all gradients."""
    Bn, N, E = x.shape
    S, G, f = A.shape[1], B.shape[2], torch.float64
    dev = x.device
    dtype = x.dtype
    xd, A = x.double(), A.double()
    pre = dt.double() + (0 if bias is None else bias.double())
    delta = torch.logaddexp(pre, torch.zeros_like(pre)) if softplus else pre
    D = torch.zeros(E, dtype=f, device=dev) if D is None else D.double()
    Bs, Cs = expand(B, E), expand(C, E)
    n = torch.full((Bn,), N, device=dev) if lengths is None else lengths.long().clamp(0, N)
    live = torch.arange(N, device=dev)[None] < n[:, None]
    mask = live[..., None]
    pre = torch.where(mask, pre, 0.0)
    xd = torch.where(mask, xd, 0.0)
    delta = torch.where(mask, delta, 0.0)
    Bs, Cs = torch.where(mask[..., None], Bs, 0.0), torch.where(mask[..., None], Cs, 0.0)
    sigma = E_DELTA + 2 * U + (N / 4 + 64) * U
    a = torch.exp(delta[..., None] * A)
    rel = RHO + (delta[..., None] * A).abs() * sigma
    ub = (delta * xd)[..., None] * Bs
    h = torch.zeros(Bn, E, S, dtype=f, device=dev) if h_in is None else h_in.double()
    hm, he = h.abs(), torch.zeros_like(h)
    hs, hms, hes, before, beforem = [], [], [], [], []
    for t in range(N):
        before.append(h)
        beforem.append(hm)
        he = a[:, t] * he + a[:, t] * hm * rel[:, t] + ub[:, t].abs() * (E_DELTA + 3 * U)
        h = a[:, t] * h + ub[:, t]
        hm = a[:, t].abs() * hm + ub[:, t].abs()
        he = he + torch.where(mask[:, t, :, None], 2 * U * hm, 0.0)
        hs.append(h)
        hms.append(hm)
        hes.append(he)
    out = dict(h=(h, he + 64 * U * hm))
    if N == 0:
        return out
    stack = lambda l: torch.stack(l, 1)
    hs, hms, hes, before, beforem = map(stack, (hs, hms, hes, before, beforem))
    s = (hs * Cs).sum(-1) + D * xd
    sm = (hms * Cs.abs()).sum(-1) + (D * xd).abs()
    se = (hes * Cs.abs()).sum(-1) + (S + 8) * U * sm
    if z is None:
        gate, gatee = torch.ones_like(s), torch.zeros_like(s)
        zd = None
    else:
        zd = torch.where(mask, z.double(), 0.0)
        sg = torch.sigmoid(zd)
        gate = zd * sg
        # (the sigmoid is a reciprocal of 1 + e^-z, flushed to 0 below 2^-126: where e^-z
        # passes 2^126 up to |z| 2^-126 of the gate is lost)
        gatee = gate.abs() * 16 * U + (zd * gate).abs() * 4 * U + zd.abs() * 2.0 ** -126
    y = s * gate
    out["y"] = (torch.where(mask, y, 0.0), se * gate.abs() + sm * gatee + half_ulp(y, dtype) + 1e-37)
    if dy is None:
        return out
    dyd = torch.where(mask, dy.double(), 0.0)
    ds = dyd * gate
    g = torch.zeros(Bn, E, S, dtype=f, device=dev) if dh_out is None else dh_out.double()
    gm, ge = g.abs(), torch.zeros_like(g)
    gs, gms, ges = [None] * N, [None] * N, [None] * N
    for t in range(N - 1, -1, -1):
        c = ds[:, t, :, None] * Cs[:, t]
        g, gm = g + c, gm + c.abs()
        ge = ge + c.abs() * 32 * U + 2 * U * gm
        gs[t], gms[t], ges[t] = g, gm, ge
        ge = a[:, t] * ge + a[:, t] * gm * rel[:, t]
        g, gm = a[:, t] * g, a[:, t].abs() * gm
    gs, gms, ges = map(stack, (gs, gms, ges))
    ratio = lambda e, m: float((e / m.clamp(min=1e-300))[m > 1e-30].max()) if bool((m > 1e-30).any()) else 0.0
    R = ratio(hes, hms) + ratio(ges, gms) + 2 * RHO + 128 * U
    chain = (128 + E / 16 + Bn * N / 32 + 2 * S) * U
    K = R + chain + float(rel.max())
    p, pm = a * before, a.abs() * beforem
    gp, gpm = gs * p, gms * pm
    q, qm = (gs * Bs).sum(-1), (gms * Bs.abs()).sum(-1)
    r, rm = (gp * A).sum(-1), (gpm * A.abs()).sum(-1)
    sp = torch.sigmoid(pre) if softplus else torch.ones_like(pre)
    ddt = torch.where(mask, (xd * q + r) * sp, 0.0)
    ddtm = torch.where(mask, ((xd.abs() * qm) + rm) * sp, 0.0)

    def put(name, v, m, dtype):
        out[name] = (v, K * m + half_ulp(v, dtype) + 1e-30)

    put("dx", delta * q + D * ds, delta.abs() * qm + (D * ds).abs(), dtype)
    put("ddt", ddt, ddtm * (1 + (0 if not softplus else 8 * U * pre.abs())), dtype)
    if zd is not None:
        put("dz", dyd * s * sg * (1 + zd * (1 - sg)), dyd.abs() * sm * sg * (1 + zd.abs() * (1 - sg)) * (1 + zd.abs()), dtype)
    fold = lambda t: t.reshape(Bn, N, G, E // G, S).sum(3)
    put("dB", fold(gs * (delta * xd)[..., None]), fold(gms * (delta * xd).abs()[..., None]), dtype)
    put("dC", fold(hs * ds[..., None]), fold(hms * ds.abs()[..., None]), dtype)
    put("dA", (gp * delta[..., None]).sum((0, 1)), (gpm * delta.abs()[..., None]).sum((0, 1)), torch.float32)
    put("dD", (ds * xd).sum((0, 1)), (ds * xd).abs().sum((0, 1)), torch.float32)
    put("ddt_bias", ddt.sum((0, 1)), ddtm.sum((0, 1)), torch.float32)
    put("dh_in", g, gm, torch.float32)
    return out


def conv(x, w, b=None, silu=True, state_in=None, lengths=None, dy=None, dstate_out=None):
    """{name: (value, bound)} of y and state, with dy of the gradients.  Sums of W
    + 1 terms, silu within 16 u (and 4 u |pre| of its exponent) and sums over
    tokens of at most 64 a thread and B N / 32 + 96 parts."""
    Bn, N, E = x.shape
    W, f, dtype = w.shape[1], torch.float64, x.dtype
    n = [N] * Bn if lengths is None else [min(max(int(v), 0), N) for v in lengths.tolist()]
    w = w.double()
    first = torch.zeros(Bn, W - 1, E, dtype=f, device=x.device) if state_in is None else state_in.double()
    xd = x.double().clone()
    live = torch.zeros(Bn, N, 1, dtype=torch.bool, device=x.device)
    for i in range(Bn):
        xd[i, n[i]:] = 0
        live[i, :n[i]] = True
    seq = torch.cat([first, xd], 1)
    pre = torch.zeros(Bn, N, E, dtype=f, device=x.device) + (0 if b is None else b.double())
    mag = pre.abs()
    for k in range(W):
        pre = pre + w[:, k] * seq[:, k:k + N]
        mag = mag + (w[:, k] * seq[:, k:k + N]).abs()
    out = {}
    sg = torch.sigmoid(pre)
    y = torch.where(live, pre * sg if silu else pre, 0.0)
    out["y"] = (y, mag * (2 * W + 24 + 4 * pre.abs()) * U + half_ulp(y, dtype) + 1e-37)
    state = torch.stack([seq[i, n[i]:n[i] + W - 1] for i in range(Bn)]) if Bn else first
    out["state"] = (state, torch.zeros_like(state))
    if dy is None:
        return out
    d1 = sg * (1 + pre * (1 - sg)) if silu else torch.ones_like(pre)
    d1m = sg * (1 + pre.abs() * (1 - sg)) + mag if silu else torch.ones_like(pre)  # |silu''| <= 1/2
    dyd = dy.double()
    d = torch.where(live, dyd * d1, 0.0)
    dm = torch.where(live, dyd.abs() * d1m * (1 + pre.abs()), 0.0)
    dseq, dseqm = torch.zeros_like(seq), torch.zeros_like(seq)
    K = (2 * W + 64 + 64 + Bn * N / 32 + 96) * U
    dw, dwm = torch.zeros_like(w), torch.zeros_like(w)
    for k in range(W):
        dseq[:, k:k + N] += w[:, k] * d
        dseqm[:, k:k + N] += w[:, k].abs() * dm
        dw[:, k] = (d * seq[:, k:k + N]).sum((0, 1))
        dwm[:, k] = (dm * seq[:, k:k + N].abs()).sum((0, 1))
    if dstate_out is not None:
        for i in range(Bn):
            dseq[i, n[i]:n[i] + W - 1] += dstate_out[i].double()
            dseqm[i, n[i]:n[i] + W - 1] += dstate_out[i].double().abs()

    def put(name, v, m, dtype):
        out[name] = (v, K * m + half_ulp(v, dtype) + 1e-37)

    put("dx", dseq[:, W - 1:], dseqm[:, W - 1:], dtype)
    put("dstate_in", dseq[:, :W - 1], dseqm[:, :W - 1], dtype)
    put("dw", dw, dwm, torch.float32)
    put("db", d.sum((0, 1)), dm.sum((0, 1)), torch.float32)
    return out


def check(name, got, want):
    value, bound = want
    assert got.shape == value.shape, f"{name}: {tuple(got.shape)} for {tuple(value.shape)}"
    err = (got.double() - value).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} off, error {float(err[bad].max()):.3e} "
                                 f"for a bound of {float(bound[bad].min()):.3e}")
