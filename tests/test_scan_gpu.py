"""GPU tests of the selective scan (prompt, one token, gradients) against the
recurrence in 64 bits; the bounds are derived in tests/ssm_reference.py."""
import math

import pytest
import torch

from tests import ssm_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0, dtype=F32):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def problem(seed, B, N, E, S, G=1, dtype=BF16, gate=True, state=True, ragged=False, skip=True, bias=True):
    """(positional arguments, keyword arguments) of a scan."""
    g = gen(seed)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(E, generator=g, device="cuda"))
    A = -(1.0 + torch.arange(S, device="cuda")) * (0.5 + torch.rand(E, S, generator=g, device="cuda"))
    args = [rand(g, B, N, E, dtype=dtype), rand(g, B, N, E, scale=0.5, dtype=dtype), A,
            rand(g, B, N, G, S, dtype=dtype), rand(g, B, N, G, S, dtype=dtype)]
    kw = dict(D=rand(g, E) if skip else None, z=rand(g, B, N, E, dtype=dtype) if gate else None,
              dt_bias=step + torch.log(-torch.expm1(-step)) if bias else None,
              h_in=rand(g, B, E, S) if state else None, lengths=None)
    if ragged:
        n = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = N
        if B > 1:
            n[1] = 0
        kw["lengths"] = n
    return args, kw


def want(args, kw, **more):
    k = dict(kw)
    k["bias"] = k.pop("dt_bias")
    return ref.scan(*args, **k, **more)


def check_fwd(R, args, kw, w=None):
    y, h = R.selective_scan_fwd(*args, **kw)
    w = want(args, kw) if w is None else w
    if args[0].numel():
        ref.check("y", y, w["y"])
    ref.check("h", h, w["h"])
    return y, h


def check_bwd(R, args, kw, dy, dh_out=None):
    w = want(args, kw, dy=dy, dh_out=dh_out)
    got = R.selective_scan_bwd(*args, dy, dh_out=dh_out, **kw)
    for name, t in got._asdict().items():
        if t is None:
            continue
        ref.check(name, t, w[name])
    assert (got.dz is None) == (kw["z"] is None) and (got.dD is None) == (kw["D"] is None)
    assert (got.ddt_bias is None) == (kw["dt_bias"] is None) and (got.dh_in is None) == (kw["h_in"] is None)
    return got


SIZES = [  # B, N, E, S, G
    (1, 1, 1, 1, 1), (2, 3, 7, 4, 1), (1, 15, 33, 5, 1), (1, 16, 32, 16, 1), (2, 17, 100, 16, 1),
    (1, 63, 64, 16, 1), (1, 64, 64, 16, 2), (2, 65, 66, 16, 3), (1, 129, 40, 8, 1), (1, 50, 300, 3, 1),
    (3, 33, 24, 11, 2), (1, 70, 20, 17, 1), (2, 40, 34, 32, 2), (1, 66, 18, 33, 1), (1, 130, 16, 64, 2),
    (2, 31, 9, 61, 3), (1, 200, 258, 16, 1), (1, 35, 130, 2, 1), (4, 20, 12, 6, 4)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,E,S,G", SIZES)
def test_forward_sizes(R, dtype, B, N, E, S, G):
    args, kw = problem(B * 7 + N * 11 + E + S, B, N, E, S, G, dtype)
    check_fwd(R, args, kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,E,S,G", SIZES)
def test_backward_sizes(R, dtype, B, N, E, S, G):
    args, kw = problem(B * 7 + N * 11 + E + S, B, N, E, S, G, dtype)
    g = gen(N)
    check_bwd(R, args, kw, rand(g, B, N, E, dtype=dtype), rand(g, B, E, S))


@pytest.mark.parametrize("gate,state,skip,bias", [(False, False, False, False), (True, False, True, False),
                                                  (False, True, False, True), (True, True, False, False)])
@pytest.mark.parametrize("softplus", [True, False])
def test_without_parts(R, gate, state, skip, bias, softplus):
    args, kw = problem(3, 2, 37, 48, 16, 1, F32, gate, state, skip=skip, bias=bias)
    if not softplus:
        # (a negative step is growth: the values, and the reference's, overflow)
        args[1] = args[1].abs() * 0.05
        if bias:
            kw["dt_bias"] = kw["dt_bias"].abs() * 0.01
    kw["softplus"] = softplus
    check_fwd(R, args, kw)
    check_bwd(R, args, kw, rand(gen(4), 2, 37, 48))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,E,S,len64", [(40, 50, 16, False), (150, 20, 64, True), (70, 96, 4, False)])
def test_padded_batch(R, dtype, N, E, S, len64):
    """Lengths of 0, N and between, beyond the range too; NaN behind them."""
    args, kw = problem(5, 6, N, E, S, 1, dtype, ragged=True)
    lengths = torch.tensor([N, 0, 1, N // 2, -3, N + 9], device="cuda")
    kw["lengths"] = lengths if len64 else lengths.int()
    for t in (args[0], args[1], args[3], args[4], kw["z"]):
        for i, n in enumerate(lengths.clamp(0, N).tolist()):
            t[i, n:] = float("nan")
    y, h = check_fwd(R, args, kw)
    assert bool((y[1] == 0).all()) and torch.equal(h[1], kw["h_in"][1])
    g = gen(6)
    dy, dh = rand(g, 6, N, E, dtype=dtype), rand(g, 6, E, S)
    dy[1:4, N // 2:] = float("nan")
    got = check_bwd(R, args, kw, dy, dh)
    assert bool((got.dx[1] == 0).all()) and torch.equal(got.dh_in[1], dh[1])


@pytest.mark.parametrize("dtype,N,E,S", [(BF16, 3000, 24, 16), (F32, 1500, 16, 16), (BF16, 1100, 8, 64)])
def test_long_sequences_with_few_channels(R, dtype, N, E, S):
    """Sequences that are cut into segments."""
    args, kw = problem(8, 1, N, E, S, 1, dtype)
    check_fwd(R, args, kw)
    check_bwd(R, args, kw, rand(gen(9), 1, N, E, dtype=dtype), rand(gen(10), 1, E, S))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_tensors(R, dtype):
    """x and z as halves of a projection, dt, B and C as slices of another, a
    sequence shared by the batch, and gradients into slices."""
    g = gen(11)
    B, N, E, S = 3, 29, 41, 16
    args, kw = problem(12, B, N, E, S, 1, dtype)
    xz = rand(g, B, N, 2 * E + 3, dtype=dtype)
    rest = rand(g, B, N, E + 2 * S + 1, scale=0.5, dtype=dtype)
    args[0], kw["z"] = xz[..., 1:E + 1], xz[..., E + 2:2 * E + 2]
    args[1] = rest[..., 1:E + 1]
    args[3], args[4] = rest[..., E + 1:E + 1 + S].unsqueeze(2), rest[..., E + 1 + S:].unsqueeze(2)
    w = want(args, kw)
    buf = torch.full((B, N, 3 * E), 7.0, dtype=dtype, device="cuda")
    y, h = R.selective_scan_fwd(*args, **kw, out=buf[..., E:2 * E])
    ref.check("y", y, w["y"])
    assert bool((buf[..., :E] == 7).all()) and bool((buf[..., 2 * E:] == 7).all())
    # [B, N, S] without the groups' dimension
    y3, _ = R.selective_scan_fwd(*args[:3], args[3].squeeze(2), args[4].squeeze(2), **kw)
    assert torch.equal(y3, y)
    shared = [args[0][:1].expand(B, -1, -1), *args[1:]]
    check_fwd(R, shared, kw)
    dy = rand(g, B, N, E, dtype=dtype)
    plain = check_bwd(R, args, kw, dy)
    dxz = torch.full((B, N, 2 * E + 1), 7.0, dtype=dtype, device="cuda")
    got = R.selective_scan_bwd(*args, dy, **kw, dx=dxz[..., :E], dz=dxz[..., E + 1:])
    assert torch.equal(got.dx, plain.dx) and torch.equal(got.dz, plain.dz)
    assert bool((dxz[..., E] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,E,S,G", [(1, 1, 1, 1), (3, 50, 16, 2), (2, 33, 7, 1), (70, 300, 16, 1),
                                     (5, 40, 64, 4), (300, 640, 4, 1), (9, 20, 33, 1), (64, 1024, 32, 2)])
def test_step(R, dtype, B, E, S, G):
    args, kw = problem(B + E, B, 1, E, S, G, dtype)
    w = want(args, kw)
    one = [args[0][:, 0], args[1][:, 0], args[2], args[3][:, 0], args[4][:, 0]]
    h = kw["h_in"].clone()
    opt = dict(D=kw["D"], z=kw["z"][:, 0], dt_bias=kw["dt_bias"])
    out = torch.empty_like(h)
    y = R.selective_scan_step(*one, h, h_out=out, **opt)
    assert torch.equal(h, kw["h_in"])
    ref.check("y", y[:, None], w["y"])
    ref.check("h", out, w["h"])
    y2 = R.selective_scan_step(*one, h, **opt)  # in place
    assert torch.equal(y, y2) and torch.equal(h, out)


def test_prompt_then_tokens(R):
    """A prompt in two parts and tokens one by one are the whole sequence."""
    args, kw = problem(20, 2, 60, 48, 16, 2, F32)
    w = want(args, kw)
    part = lambda a, b: [args[0][:, a:b], args[1][:, a:b], args[2], args[3][:, a:b], args[4][:, a:b]]
    opt = dict(D=kw["D"], dt_bias=kw["dt_bias"])
    y1, h = R.selective_scan_fwd(*part(0, 20), z=kw["z"][:, :20], h_in=kw["h_in"], **opt)
    y2, h = R.selective_scan_fwd(*part(20, 50), z=kw["z"][:, 20:50], h_in=h, **opt)
    ys = [y1, y2]
    for t in range(50, 60):
        one = [v if v is args[2] else v[:, 0] for v in part(t, t + 1)]
        ys.append(R.selective_scan_step(*one, h, z=kw["z"][:, t], **opt)[:, None])
    ref.check("y", torch.cat(ys, 1), w["y"])
    ref.check("h", h, w["h"])


@pytest.mark.parametrize("B,N", [(2, 0), (0, 5), (0, 0)])
def test_nothing_to_do(R, B, N):
    args, kw = problem(21, B, N, 10, 16, 1, F32)
    y, h = R.selective_scan_fwd(*args, **kw)
    assert y.shape == (B, N, 10)
    assert torch.equal(h, kw["h_in"])
    dh = rand(gen(1), B, 10, 16)
    got = R.selective_scan_bwd(*args, torch.empty_like(args[0]), dh_out=dh, **kw)
    assert torch.equal(got.dh_in, dh)
    assert all(float(t.abs().max()) == 0 for t in (got.dA, got.dD, got.ddt_bias))


def test_large_steps_and_gates(R):
    """Steps that forget everything, steps of nearly nothing, closed gates."""
    args, kw = problem(22, 1, 40, 32, 16, 1, F32)
    args[1][:, ::5] = 60.0
    args[1][:, 1::5] = -60.0
    kw["z"][:, ::3] = -90.0
    kw["z"][:, 1::7] = 90.0
    y, _ = check_fwd(R, args, kw)
    assert bool(torch.isfinite(y).all())
    check_bwd(R, args, kw, rand(gen(23), 1, 40, 32))


def test_nan_stays_in_its_channel_and_sequence(R):
    args, kw = problem(24, 2, 50, 40, 16, 1, F32)
    args[0][1, 20, 7] = float("nan")
    y, h = R.selective_scan_fwd(*args, **kw)
    bad = torch.isnan(y)
    assert bool(bad[1, 20:, 7].all()) and bool(torch.isnan(h[1, 7]).all())
    bad[1, 20:, 7] = False
    assert not bool(bad.any())


def test_equal_calls_give_equal_bits(R):
    args, kw = problem(25, 2, 300, 200, 16, 1, BF16)
    dy = rand(gen(26), 2, 300, 200, dtype=BF16)
    first = (*R.selective_scan_fwd(*args, **kw), *R.selective_scan_bwd(*args, dy, **kw))
    for _ in range(3):
        again = (*R.selective_scan_fwd(*args, **kw), *R.selective_scan_bwd(*args, dy, **kw))
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_gradients_against_differences(R):
    """sum(dy y) + sum(dh h) along random directions of every input: central
    five-point differences with step 0.02 (truncation h^4 / 30 of the fifth
    derivative, below 1e-6 of it; rounding 1.5 u sum|dy y| / h = 1e-5 of a sum
    ten times the derivative's size) within 2e-3 of the derivatives' size."""
    args, kw = problem(27, 2, 23, 12, 5, 2, F32)
    g = gen(28)
    dy, dh = rand(g, 2, 23, 12), rand(g, 2, 12, 5)
    grads = R.selective_scan_bwd(*args, dy, dh_out=dh, **kw)

    def loss(args, kw):
        y, h = R.selective_scan_fwd(*args, **kw)
        return float((dy.double() * y.double()).sum() + (dh.double() * h.double()).sum())

    step = 0.02
    for name in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h_in"):
        pos = ("x", "dt", "A", "B", "C").index(name) if name in ("x", "dt", "A", "B", "C") else None
        base = args[pos] if pos is not None else kw[name]
        grad = getattr(grads, "d" + name).double()
        v = rand(g, *base.shape)
        if name == "A":
            v = v * 0.2
        f = []
        for k in (-2, -1, 1, 2):
            a2, k2 = list(args), dict(kw)
            moved = base + k * step * v
            if pos is not None:
                a2[pos] = moved
            else:
                k2[name] = moved
            f.append(loss(a2, k2))
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * step)
        size = float((grad * v.double()).norm())
        assert abs(fd - float((grad * v.double()).sum())) <= 2e-3 * max(size, 1.0), name


def test_other_stream_and_graph(R):
    args, kw = problem(29, 2, 400, 64, 16, 1, BF16)
    dy = rand(gen(30), 2, 400, 64, dtype=BF16)
    call = lambda **k: (*R.selective_scan_fwd(*args, **kw, **k), *R.selective_scan_bwd(*args, dy, **kw, **k))
    first = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        t.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("S", [3, 16, 64])
@pytest.mark.parametrize("prompt", [False, True])
def test_decays_at_the_end_of_the_normal_numbers(R, prompt, S):
    """x = 0, so that the state is the decayed one alone.  The exponent delta A log2(e) has
    three roundings (the constant, A log2(e), its product with delta), each 2^-24 of |w| <= 131,
    the exponential 2^-22 of itself; below 2^-126 it counts as 0, 2^-126 of the state at most."""
    E, U = 40, 2.0 ** -24
    shape = (2, 1, E) if prompt else (2, E)
    x, dt = torch.zeros(shape, device="cuda"), torch.ones(shape, device="cuda")
    A = -(math.log(2) * torch.linspace(121, 131, S, device="cuda")).expand(E, S).contiguous()
    B = torch.ones(*shape[:-1], 1, S, device="cuda")
    h0 = rand(gen(31), 2, E, S)
    if prompt:
        _, h = R.selective_scan_fwd(x, dt, A, B, B, softplus=False, h_in=h0)
    else:
        h = torch.empty_like(h0)
        R.selective_scan_step(x, dt, A, B, B, h0, softplus=False, h_out=h)
    want = torch.exp(A.double()) * h0.double()
    rel = 3 * U * A.double().abs() + 8 * U
    # (a product of a decay above 2^-126 and |h0| < 1 is rounded to 2^-149)
    bound = want.abs() * rel + 2.0 ** -126 * (1 + rel) * h0.double().abs() + 2.0 ** -149
    assert bool(((h.double() - want).abs() <= bound).all())
    low = A.double() / math.log(2) < -126.1
    assert bool((h[low.expand_as(h)] == 0).all())
    assert bool((h[(A.double() / math.log(2) > -125.9).expand_as(h)] != 0).all())
