"""GPU tests of the causal convolution and its gradients against the sums in 64
bits; the bounds are derived in tests/ssm_reference.py."""
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


def check(R, x, w, b, dy, state_in=None, dstate_out=None, lengths=None, silu=True):
    want = ref.conv(x, w, b, silu, state_in, lengths, dy, dstate_out)
    y, state = R.causal_conv_fwd(x, w, b, silu=silu, state_in=state_in, lengths=lengths)
    ref.check("y", y, want["y"])
    assert torch.equal(state.double(), want["state"][0])
    dx, dw, db, ds = R.causal_conv_bwd(x, w, b, dy, silu=silu, state_in=state_in, dstate_out=dstate_out, lengths=lengths)
    ref.check("dx", dx, want["dx"])
    ref.check("dw", dw, want["dw"])
    assert (db is None) == (b is None) and (ds is None) == (state_in is None)
    if b is not None:
        ref.check("db", db, want["db"])
    if state_in is not None:
        ref.check("dstate_in", ds, want["dstate_in"])
    return y, state, dx, dw, db, ds


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("B,N,E", [(1, 1, 1), (2, 2, 8), (1, 3, 7), (3, 4, 16), (1, 5, 33), (2, 63, 40), (1, 64, 24),
                                   (2, 65, 12), (1, 500, 104), (5, 131, 20)])
def test_sizes(R, dtype, W, B, N, E):
    g = gen(B * 100 + N * 7 + E + W)
    x, dy = rand(g, B, N, E, dtype=dtype), rand(g, B, N, E, dtype=dtype)
    w, b = rand(g, E, W, scale=0.5), rand(g, E, scale=0.1)
    state, ds = rand(g, B, W - 1, E, dtype=dtype), rand(g, B, W - 1, E, dtype=dtype)
    check(R, x, w, b, dy, state, ds)


@pytest.mark.parametrize("bias,state,silu", [(False, False, True), (True, False, False), (False, True, False)])
def test_without_parts(R, bias, state, silu):
    g = gen(1)
    x, dy = rand(g, 2, 40, 32), rand(g, 2, 40, 32)
    check(R, x, rand(g, 32, 4), rand(g, 32) if bias else None, dy, rand(g, 2, 3, 32) if state else None, None, None, silu)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W,E,len64", [(4, 16, False), (3, 9, True), (2, 40, False)])
def test_padded_batch(R, dtype, W, E, len64):
    """Lengths shorter than the taps, 0 and beyond the range; NaN behind them."""
    N = 90
    g = gen(2)
    lengths = torch.tensor([N, 0, 1, 2, 3, 47, -1, N + 5], device="cuda")
    x, dy = rand(g, 8, N, E, dtype=dtype), rand(g, 8, N, E, dtype=dtype)
    for i, n in enumerate(lengths.clamp(0, N).tolist()):
        x[i, n:] = float("nan")
        dy[i, n:] = float("nan")
    state, ds = rand(g, 8, W - 1, E, dtype=dtype), rand(g, 8, W - 1, E, dtype=dtype)
    y, after, dx, *_ = check(R, x, rand(g, E, W), rand(g, E), dy, state, ds, lengths if len64 else lengths.int())
    assert bool((y[1] == 0).all()) and torch.equal(after[1], state[1]) and bool((dx[6] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows(R, dtype):
    g = gen(3)
    wide = rand(g, 3, 50, 70, dtype=dtype)
    w, b = rand(g, 33, 4), rand(g, 33)
    dy = rand(g, 3, 50, 40, dtype=dtype)[..., 3:36]
    x = wide[..., 5:38]
    y, state, dx, dw, db, _ = check(R, x, w, b, dy)
    buf = torch.full((3, 50, 70), 7.0, dtype=dtype, device="cuda")
    assert torch.equal(R.causal_conv_fwd(x, w, b, out=buf[..., 30:63])[0], y)
    assert bool((buf[..., :30] == 7).all()) and bool((buf[..., 63:] == 7).all())
    got = R.causal_conv_bwd(x, w, b, dy, dx=buf[..., 30:63])
    assert torch.equal(got[0], dx) and bool((buf[..., :30] == 7).all())
    check(R, x[:1].expand(3, -1, -1), w, b, dy)
    check(R, wide.transpose(0, 1)[..., 5:38], w, b, dy.transpose(0, 1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,E,W", [(1, 1, 4), (3, 40, 4), (2, 33, 3), (17, 64, 2), (300, 520, 4)])
def test_step(R, dtype, B, E, W):
    g = gen(B + E)
    x, w, b = rand(g, B, E, dtype=dtype), rand(g, E, W), rand(g, E)
    state = rand(g, B, W - 1, E, dtype=dtype)
    want = ref.conv(x[:, None], w, b, True, state)
    after = torch.empty_like(state)
    kept = state.clone()
    y = R.causal_conv_step(x, w, b, state, state_out=after)
    assert torch.equal(state, kept)
    ref.check("y", y[:, None], want["y"])
    assert torch.equal(after.double(), want["state"][0])
    assert torch.equal(R.causal_conv_step(x, w, b, state), y) and torch.equal(state, after)  # in place


def test_parts_are_the_whole(R):
    g = gen(5)
    x, w, b = rand(g, 2, 30, 24), rand(g, 24, 4), rand(g, 24)
    y, state = R.causal_conv_fwd(x, w, b)
    a, s = R.causal_conv_fwd(x[:, :2], w, b)
    c, s = R.causal_conv_fwd(x[:, 2:25], w, b, state_in=s, state_out=s)
    rest = [R.causal_conv_step(x[:, t], w, b, s)[:, None] for t in range(25, 30)]
    assert torch.equal(torch.cat([a, c, *rest], 1), y) and torch.equal(s, state)


@pytest.mark.parametrize("B,N", [(2, 0), (0, 5)])
def test_nothing_to_do(R, B, N):
    g = gen(6)
    x, w, b = rand(g, B, N, 8), rand(g, 8, 4), rand(g, 8)
    s = rand(g, B, 3, 8)
    y, state = R.causal_conv_fwd(x, w, b, state_in=s)
    assert y.shape == x.shape and torch.equal(state, s)
    _, dw, db, ds = R.causal_conv_bwd(x, w, b, x, state_in=s, dstate_out=s)
    assert torch.equal(ds, s) and float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_gradients_against_differences(R):
    """Five-point differences of sum(dy y) + sum(ds state), step 0.02 (truncation
    below 1e-6 of the fifth derivative, rounding 1e-5 of the sum), within 2e-3 of
    the derivatives' size."""
    g = gen(7)
    x, w, b, s = rand(g, 2, 9, 6), rand(g, 6, 4), rand(g, 6), rand(g, 2, 3, 6)
    dy, ds = rand(g, 2, 9, 6), rand(g, 2, 3, 6)
    grads = R.causal_conv_bwd(x, w, b, dy, state_in=s, dstate_out=ds)

    def loss(x, w, b, s):
        y, after = R.causal_conv_fwd(x, w, b, state_in=s)
        return float((dy.double() * y.double()).sum() + (ds.double() * after.double()).sum())

    for i, grad in enumerate(grads):
        args = [x, w, b, s]
        v = rand(g, *args[i].shape)
        f = []
        for k in (-2, -1, 1, 2):
            moved = list(args)
            moved[i] = args[i] + k * 0.02 * v
            f.append(loss(*moved))
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / 0.24
        d = grad.double() * v.double()
        assert abs(fd - float(d.sum())) <= 2e-3 * max(float(d.norm()), 1.0)


def test_equal_bits_other_stream_and_graph(R):
    g = gen(8)
    x, dy, w, b = rand(g, 3, 700, 128, dtype=BF16), rand(g, 3, 700, 128, dtype=BF16), rand(g, 128, 4), rand(g, 128)
    call = lambda **k: (*R.causal_conv_fwd(x, w, b, **k), *R.causal_conv_bwd(x, w, b, dy, **k)[:3])
    first = call()
    assert all(torch.equal(p, q) for p, q in zip(first, call()))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for t in got:
        t.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, got))
