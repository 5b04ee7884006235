"""GPU tests of the RMS norm with the residual's addition, its 8-bit output and
its gradients against the formulas in 64 bits.

Tolerances, u = 2^-24: the mean square is a sum of positive terms in chains of
at most 64 a thread (rows up to 16384; d / 1024 beyond) and 10 joins, and rstd
half as far off: 40 u, 3 u for its root and two products: 64 u of |y| (128 u for
longer rows).  h is one rounding of the sum.  The gradients' row sum has chains
as long, of terms that carry rstd's error: 128 u of sum |g n|; dw: chains of
at most rows / 152 + 64 rows and 1300 parts in warps of 32 (96 joins).
An e4m3 value is y / scale, within 70 u of the exact quotient, rounded to
nearest: off by half a step of e4m3 (2^-4 of itself, 2^-10 below its normal
range, where values are multiples of 2^-9) and those 70 u.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


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


def half(ref, dtype):
    return ref.abs() * 2.0 ** -8 if dtype == BF16 else ref.abs() * U


def kept(x, r):
    """The sum as it is kept: both types hold the operands exactly, and fp32's sum
    of two bf16 values rounds once more only below fp32's last bit."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def normed(h, w, eps):
    f = h.double()
    rstd = 1.0 / torch.sqrt((f * f).mean(-1) + eps)
    y = f * rstd[..., None]
    return rstd, y if w is None else y * w.double()


def units(d):
    return 64 * U if d <= 16384 else (64 + d / 1024) * U


def check_fwd(R, x, r, w, eps=1e-5):
    y, h, rstd = R.rmsnorm_fwd(x, w, residual=r, eps=eps)
    want = kept(x, r)
    assert torch.equal(h, want) and y.dtype == x.dtype
    rr, ry = normed(want, w, eps)
    k = units(x.shape[-1])
    assert bool(((rstd.double() - rr).abs() <= k * rr).all())
    assert bool(((y.double() - ry).abs() <= k * ry.abs() + half(ry, x.dtype) + 1e-37).all())
    return y, h, rstd


def check_bwd(R, h, dy, dh, w, rstd):
    dx, dw = R.rmsnorm_bwd(h, dy, w, rstd, dh=dh)
    f, q, r = h.double(), dy.double(), rstd.double()[..., None]
    n, g = f * r, q if w is None else q * w.double()
    mean, meanm = (g * n).mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    want = r * (g - n * mean)
    mag = r * (g.abs() + n.abs() * meanm)
    if dh is not None:
        want, mag = want + dh.double(), mag + dh.double().abs()
    k = 2 * units(h.shape[-1])
    assert bool(((dx.double() - want).abs() <= k * mag + half(want, h.dtype) + 1e-37).all())
    lead = tuple(range(h.dim() - 1))
    rows = h.numel() // max(h.shape[-1], 1)
    tol = (rows / 152 + 64 + 96) * U * (q * n).abs().sum(lead) + 1e-37
    assert bool(((dw.double() - (q * n).sum(lead)).abs() <= tol).all())
    return dx, dw


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", [
    (1, 1), (3, 2), (5, 7), (2, 31), (7, 32), (9, 33), (4, 64), (33, 255), (17, 256), (3, 264), (3, 513),
    (11, 1000), (300, 1024), (5, 1537), (70, 2048), (3, 2049), (1, 4096), (700, 4096), (2, 4104), (3, 8191),
    (40, 8192), (2, 8200), (3, 10007), (20, 16384), (2, 16392), (1, 40000), (2, 70001)])
def test_sizes(R, dtype, rows, d):
    g = gen(rows * 1009 + d)
    x, r, w = rand(g, rows, d, dtype=dtype), rand(g, rows, d, scale=2.0, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    dy, dh = rand(g, rows, d, scale=0.1, dtype=dtype), rand(g, rows, d, scale=0.1, dtype=dtype)
    _, h, rstd = check_fwd(R, x, r, w)
    check_bwd(R, h, dy, dh, w, rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d", [(30000, 64), (20011, 100), (3000, 768)])
def test_many_short_rows(R, dtype, rows, d):
    g = gen(rows)
    x, w, dy = rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1), rand(g, rows, d, dtype=dtype)
    _, h, rstd = check_fwd(R, x, None, w)
    assert h.data_ptr() == x.data_ptr()
    check_bwd(R, h, dy, None, w, rstd)


def test_without_gain_or_residual(R):
    g = gen(1)
    x, r, dy = rand(g, 6, 264, dtype=BF16), rand(g, 6, 264, dtype=BF16), rand(g, 6, 264, dtype=BF16)
    for res in (None, r):
        _, h, rstd = check_fwd(R, x, res, None, eps=0.0)
        check_bwd(R, h, dy, res, None, rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows(R, dtype):
    g = gen(2)
    w = 1.0 + rand(g, 96, scale=0.1)
    for x in (rand(g, 4, 5, 131, dtype=dtype)[..., 3:99], rand(g, 4, 5, 96, dtype=dtype).transpose(0, 1),
              rand(g, 2, 3, 4, 5, 104, dtype=dtype)[..., :96], rand(g, 1, 5, 96, dtype=dtype).expand(4, 5, 96)):
        r, dy = (rand(g, *x.shape[:-1], 100, dtype=dtype)[..., 1:97] for _ in range(2))
        _, h, rstd = check_fwd(R, x, r if x.dim() == 3 else None, w)
        check_bwd(R, h, dy, r if x.dim() == 3 else None, w, rstd)
    buf = torch.full((4, 5, 131), 7.0, dtype=dtype, device="cuda")
    x = rand(g, 4, 5, 96, dtype=dtype)
    # (off the 16-byte boundary the sums have another order: the formulas' tolerance, not equal bits)
    y = R.rmsnorm_fwd(x, w, out=buf[..., 3:99])[0]
    ry = normed(x, w, 1e-5)[1]
    assert bool(((y.double() - ry).abs() <= units(96) * ry.abs() + half(ry, dtype) + 1e-37).all())
    assert bool((buf[..., :3] == 7).all()) and bool((buf[..., 99:] == 7).all())


@pytest.mark.parametrize("d", [96, 97, 4096, 20000])
def test_in_place(R, d):
    """h over x or the residual, y over the other, dx over any input."""
    g = gen(3)
    x, r, dy, dh, w = rand(g, 9, d), rand(g, 9, d), rand(g, 9, d), rand(g, 9, d), rand(g, d)
    y, h, rstd = R.rmsnorm_fwd(x, w, residual=r)
    for swap in (False, True):
        a, b = x.clone(), r.clone()
        over, other = (b, a) if swap else (a, b)
        got = R.rmsnorm_fwd(a, w, residual=b, residual_out=over, out=other)
        assert torch.equal(got[0], y) and torch.equal(got[1], h) and got[1] is over
    a = x.clone()
    assert torch.equal(R.rmsnorm_fwd(a, w, out=a)[0], R.rmsnorm_fwd(x, w)[0])
    want = R.rmsnorm_bwd(h, dy, w, rstd, dh=dh)
    for i in range(3):
        t = [h.clone(), dy.clone(), dh.clone()]
        got = R.rmsnorm_bwd(t[0], t[1], w, rstd, dh=t[2], dx=t[i])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_zero_rows_and_nan_rows(R):
    g = gen(4)
    x, w = rand(g, 5, 300), rand(g, 300)
    x[1] = 0.0
    x[3, 17] = float("nan")
    y, _, rstd = R.rmsnorm_fwd(x, w)
    assert bool((y[1] == 0).all()) and bool(torch.isnan(y[3]).all()) and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 64 * U
    _, ry = normed(x, w, 1e-5)
    ok = [0, 2, 4]
    assert bool(((y.double() - ry)[ok].abs() <= 64 * U * ry[ok].abs() + half(ry[ok], F32)).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d,group", [(3, 64, 0), (5, 100, 0), (4, 256, 128), (7, 1000, 128), (2, 4096, 128),
                                          (9, 33, 8), (600, 512, 128), (3, 8192, 128), (2, 16384, 0), (3, 5001, 128),
                                          (2, 20000, 128), (1, 20001, 0), (2, 40000, 2048), (6, 128, 4096)])
def test_quant(R, dtype, rows, d, group):
    g = gen(rows + d + group)
    x, r, w = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    x[0, :8] = 0
    r[0, :8] = 0
    q, scales, h = R.rmsnorm_quant(x, w, residual=r, group=group)
    assert torch.equal(h, kept(x, r)) and q.dtype == torch.float8_e4m3fn
    size = min(group or d, d)
    _, y = normed(h, w, 1e-5)
    blocks = list(y.split(size, -1))
    want = torch.stack([b.abs().amax(-1) for b in blocks], -1) / 448.0
    k = units(d) + 4 * U
    assert scales.shape == want.shape and bool(((scales.double() - want).abs() <= k * want).all())
    for i, (b, v) in enumerate(zip(blocks, q.float().split(size, -1))):
        s = scales[..., i:i + 1].double()
        exact = torch.where(s > 0, b / s.clamp(min=1e-300), 0.0)
        tol = (exact.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + exact.abs() * (k + 6 * U)
        assert bool(((v.double() - exact).abs() <= tol).all())
        assert float(v.abs().max()) == 448.0 or float(s.max()) == 0.0


def test_quant_of_zero_and_tiny_rows(R):
    x = torch.zeros(3, 256, device="cuda")
    x[1, 5] = 1e-30
    x[2, :128] = 3e38
    q, scales, _ = R.rmsnorm_quant(x, group=128, eps=0.5)
    assert bool((q[0].float() == 0).all()) and bool((scales[0] == 0).all())
    assert bool(torch.isfinite(q[1].float()).all()) and float(q[1, 5].float()) == 448.0
    assert bool((scales[1, 1] == 0)) and bool((q[2].float() == 0).all())  # (3e38^2 is infinite: rstd 0)


def test_strided_quant(R):
    g = gen(5)
    x = rand(g, 4, 5, 131, dtype=BF16)[..., 3:99]
    q, s, _ = R.rmsnorm_quant(x, group=32)
    buf = torch.zeros(4, 5, 200, dtype=torch.uint8, device="cuda").fill_(9)
    out = buf[..., 7:103].view(torch.float8_e4m3fn)
    q2, s2, _ = R.rmsnorm_quant(x, group=32, out=out)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s, s2)
    assert bool((buf[..., :7] == 9).all()) and bool((buf[..., 103:] == 9).all())


def test_no_rows(R):
    x = torch.empty(0, 40, dtype=BF16, device="cuda")
    y, h, rstd = R.rmsnorm_fwd(x)
    dw = torch.full((40,), 3.0, device="cuda")
    R.rmsnorm_bwd(h, x, None, rstd, dw=dw)
    assert y.shape == (0, 40) and float(dw.abs().max()) == 0
    assert R.rmsnorm_quant(x, group=8)[1].shape == (0, 5)


def test_gradient_against_differences(R):
    """sum(dy y + dh h) along random directions: five-point differences, step
    0.02 (truncation below 1e-6 of the fifth derivative, rounding 1e-5 of the
    sum), within 1e-3 of ten times the derivatives' size."""
    g = gen(6)
    x, r, w, dy, dh = rand(g, 7, 130), rand(g, 7, 130), rand(g, 130), rand(g, 7, 130), rand(g, 7, 130)
    _, h, rstd = R.rmsnorm_fwd(x, w, residual=r)
    dx, dw = R.rmsnorm_bwd(h, dy, w, rstd, dh=dh)

    def loss(x, r, w):
        y, h, _ = R.rmsnorm_fwd(x, w, residual=r)
        return float((dy.double() * y.double()).sum() + (dh.double() * h.double()).sum())

    for i, grad in ((0, dx), (1, dx), (2, dw)):
        args = [x, r, w]
        v = rand(g, *args[i].shape)
        f = []
        for k in (-2, -1, 1, 2):
            moved = list(args)
            moved[i] = args[i] + k * 0.02 * v
            f.append(loss(*moved))
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / 0.24
        d = grad.double() * v.double()
        assert abs(fd - float(d.sum())) <= 1e-2 * float(d.norm())


def test_equal_bits_other_stream_and_graph(R):
    g = gen(7)
    x, r, dy, w = (rand(g, 3000, 512, dtype=BF16) for _ in range(3)), None, None, rand(g, 512)
    x, r, dy = x
    _, h, rstd = R.rmsnorm_fwd(x, w, residual=r)
    call = lambda **k: (*R.rmsnorm_fwd(x, w, residual=r, **k), *R.rmsnorm_bwd(h, dy, w, rstd, dh=r, **k),
                        R.rmsnorm_quant(x, w, residual=r, group=128, **k)[1])
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
