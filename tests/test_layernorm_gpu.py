"""GPU tests of LayerNorm and its gradients against the formulas in 64 bits.

Tolerances, from fp32 arithmetic with unit roundoff u = 2^-24:
  * y and dx: the mean and the row sums are added in chains of at most 64
    terms a thread and 10 joins, so their relative error is below 80 u of the
    sum of magnitudes; a row's level is at most 4 standard deviations here, and
    the remaining steps add a few u each: 512 u = 3.1e-5 of the largest value;
  * a bf16 result adds half an ulp of itself;
  * dw, db: chains of at most 64 rows and 64 partial sums and a relative error
    of h of 100 u (its row's mean): 256 u of the sum of |dy h| or |dy|.
"""
import pytest
import torch

from tests.helpers import bf16_half_ulp

pytestmark = pytest.mark.gpu
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


def rand(g, *shape, scale=1.0, dtype=torch.float32):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def ref_fwd(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(var + eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean[..., 0], rstd[..., 0]


def ref_bwd(x, dy, w, mean, rstd):
    x, dy, r = x.double(), dy.double(), rstd.double()[..., None]
    h = (x - mean.double()[..., None]) * r
    g = dy if w is None else dy * w.double()
    dx = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    rows = tuple(range(x.dim() - 1))
    return dx, (dy * h).sum(rows), dy.sum(rows), (dy * h).abs().sum(rows), dy.abs().sum(rows)


def close(got, ref, what):
    """512 u of the largest value, and half an ulp of a bf16 result."""
    tol = 512 * U * ref.abs().amax().clamp(min=1e-30)
    if got.dtype == torch.bfloat16:
        tol = tol + torch.from_numpy(bf16_half_ulp(ref.cpu().numpy())).to(ref.device)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{what}: {float(err.max()):.3e}"


def check(R, x, dy, w, b, eps=1e-5):
    y, mean, rstd = R.layernorm_fwd(x, w, b, eps=eps)
    ry, rm, rr = ref_fwd(x, w, b, eps)
    assert y.dtype == x.dtype and y.shape == x.shape
    if x.numel():
        close(y, ry, "y")
        scale = x.double().abs().amax()
        assert float((mean.double() - rm).abs().max()) <= 80 * U * float(scale)
        assert float(((rstd.double() - rr) / rr).abs().max()) <= 512 * U
    dx, dw, db = R.layernorm_bwd(x, dy, w, mean, rstd)
    rx, rw, rb, aw, ab = ref_bwd(x, dy, w, mean, rstd)
    assert dx.dtype == x.dtype
    if x.numel():
        close(dx, rx, "dx")
    assert bool(((dw.double() - rw).abs() <= 256 * U * aw + 1e-30).all())
    assert bool(((db.double() - rb).abs() <= 256 * U * ab + 1e-30).all())
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [
    (1, 1), (3, 2), (5, 7), (2, 31), (7, 32), (9, 33), (4, 64), (33, 255), (17, 256), (3, 513),
    (11, 1000), (300, 1024), (5, 1537), (70, 2048), (3, 2049), (1, 4096), (8, 4096), (700, 4096),
    (2, 4104), (3, 8191), (4, 8192), (2, 8200), (3, 10007), (2, 16384), (2, 16392), (1, 40000),
    (2, 70001)])
def test_sizes(R, dtype, rows, d):
    g = gen(rows * 100003 + d)
    x = rand(g, rows, d) * 1.5 + rand(g, rows, 1)
    x, dy = x.to(dtype), rand(g, rows, d, scale=0.1, dtype=dtype)
    check(R, x, dy, 1.0 + rand(g, d, scale=0.1), rand(g, d, scale=0.1))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(50000, 64), (20011, 100), (3000, 768)])
def test_many_short_rows(R, dtype, rows, d):
    g = gen(rows + d)
    x, dy = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype)
    w = 1.0 + rand(g, d, scale=0.1)
    y, mean, rstd = R.layernorm_fwd(x, w)
    close(y, ref_fwd(x, w, None, 1e-5)[0], "y")
    dx, dw, db = R.layernorm_bwd(x, dy, w, mean, rstd)
    rx, rw, rb, aw, ab = ref_bwd(x, dy, w, mean, rstd)
    close(dx, rx, "dx")
    # the chains here are longer: at most rows / 152 + 200 terms
    n = rows / 152 + 200 + 100
    assert bool(((dw.double() - rw).abs() <= n * U * aw).all())
    assert bool(((db.double() - rb).abs() <= n * U * ab).all())


@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_without_gain_or_bias(R, w, b):
    g = gen(5)
    x, dy = rand(g, 6, 264, dtype=torch.bfloat16), rand(g, 6, 264, dtype=torch.bfloat16)
    check(R, x, dy, rand(g, 264) if w else None, rand(g, 264) if b else None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows(R, dtype):
    """Rows of a wider buffer, transposed leading dimensions, four of them
    that fold, and a row broadcast over the batch."""
    g = gen(6)
    w, b = 1.0 + rand(g, 96, scale=0.1), rand(g, 96, scale=0.1)
    for x in (rand(g, 4, 5, 131, dtype=dtype)[..., 3:99],
              rand(g, 4, 5, 96, dtype=dtype).transpose(0, 1),
              rand(g, 2, 3, 4, 5, 104, dtype=dtype)[..., :96],
              rand(g, 1, 5, 96, dtype=dtype).expand(4, 5, 96)):
        dy = rand(g, *x.shape[:-1], 100, dtype=dtype)[..., 1:97]
        check(R, x, dy, w, b)
    # output rows inside a wider buffer: the columns beside them stay
    buf = torch.full((4, 5, 131), 7.0, dtype=dtype, device="cuda")
    x = rand(g, 4, 5, 96, dtype=dtype)
    y, _, _ = R.layernorm_fwd(x, w, b, out=buf[..., 3:99])
    close(y, ref_fwd(x, w, b, 1e-5)[0], "y")
    assert bool((buf[..., :3] == 7).all()) and bool((buf[..., 99:] == 7).all())


@pytest.mark.parametrize("d", [96, 97, 4096, 20000])
def test_in_place(R, d):
    """y over x, dx over dy and dx over x give the bits of separate outputs."""
    g = gen(7)
    x, dy, w = rand(g, 9, d), rand(g, 9, d), rand(g, d)
    y, mean, rstd = R.layernorm_fwd(x, w)
    x2 = x.clone()
    assert torch.equal(R.layernorm_fwd(x2, w, out=x2)[0], y)
    dx, dw, db = R.layernorm_bwd(x, dy, w, mean, rstd)
    for over in (0, 1):
        a, b = x.clone(), dy.clone()
        got = R.layernorm_bwd(a, b, w, mean, rstd, dx=(a, b)[over])
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d", [(611, 1), (611, 45), (611, 131), (611, 255), (611, 321), (611, 513),
                                    (611, 1031), (211, 4097), (13, 8193)])
def test_rows_off_the_16_byte_boundary(R, dtype, rows, d):
    """Rows that begin anywhere in a 16-byte word, x, dy and the outputs at
    different places, and what lies between the rows: NaN, and left alone."""
    g = gen(11 + d)
    w, b = 1.0 + rand(g, d, scale=0.1), rand(g, d, scale=0.1)

    def rows_at(offset, pitch, fill=float("nan")):
        flat = torch.full((rows * pitch + 16,), fill, dtype=dtype, device="cuda")
        return flat, flat[offset:offset + rows * pitch].view(rows, pitch)[:, :d]

    for ox, og, oy, pad in ((1, 2, 3, 0), (7, 0, 5, 3), (3, 3, 3, 5)):
        x, dy = rows_at(ox, d + pad)[1], rows_at(og, d + pad)[1]
        x.copy_(rand(g, rows, d))
        dy.copy_(rand(g, rows, d, scale=0.1))
        y, mean, rstd, dx, dw, db = check(R, x, dy, w, b)
        flat, out = rows_at(oy, d + 7, 5.0)
        assert torch.equal(R.layernorm_fwd(x, w, b, out=out)[0], y)
        out.fill_(5.0)
        assert bool((flat == 5.0).all())
        got = R.layernorm_bwd(x, dy, w, mean, rstd, dx=out)
        assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
        out.fill_(5.0)
        assert bool((flat == 5.0).all())
        x2 = x.clone()
        assert torch.equal(R.layernorm_fwd(x2, w, b, out=x2)[0], y)


def test_large_level_and_small_spread(R):
    """A level of 1000 standard deviations: the deviations' mean square keeps
    the variance to the rounding of x - mean (mean error 80 u of the level)."""
    g = gen(8)
    x = 1000.0 + rand(g, 5, 4096)
    y, mean, rstd = R.layernorm_fwd(x)
    ry, rm, rr = ref_fwd(x, None, None, 1e-5)
    assert float((mean.double() - rm).abs().max()) <= 80 * U * 1000
    assert float((y.double() - ry).abs().max()) <= 100 * U * 1000 * 2
    assert float(((rstd.double() - rr) / rr).abs().max()) <= (80 * U * 1000) ** 2 + 512 * U


def test_constant_rows_and_nan_rows(R):
    g = gen(9)
    x = rand(g, 6, 300)
    x[1] = 3.0
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    w, b = rand(g, 300), rand(g, 300)
    y, mean, rstd = R.layernorm_fwd(x, w, b)
    assert torch.equal(y[1], b)
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[4]).all())
    keep = [0, 1, 2, 5]
    close(y[keep], ref_fwd(x, w, b, 1e-5)[0][keep], "rows beside a NaN")


def test_no_rows(R):
    x = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = R.layernorm_fwd(x)
    assert y.shape == (0, 40)
    dw, db = torch.full((40,), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    R.layernorm_bwd(x, x, None, mean, rstd, dw=dw, db=db)
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


@pytest.mark.parametrize("dtype,rows,d", [(torch.bfloat16, 3000, 512), (torch.float32, 1000, 97)])
def test_equal_calls_give_equal_bits(R, dtype, rows, d):
    g = gen(10)
    x, dy, w = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype), rand(g, d)
    _, mean, rstd = R.layernorm_fwd(x, w)
    first = R.layernorm_bwd(x, dy, w, mean, rstd)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, R.layernorm_bwd(x, dy, w, mean, rstd)))


def test_gradient_against_differences(R):
    """sum(dy y) along random directions of x, w and b: five-point
    differences of the forward (step 0.02: truncation below h^4 = 1.6e-7 of the
    fifth derivative, rounding about 1.5 u sum|dy y| / h) within 1e-3 of the
    size of the derivatives."""
    g = gen(11)
    x, dy, w, b = rand(g, 7, 130), rand(g, 7, 130), rand(g, 130), rand(g, 130)
    _, mean, rstd = R.layernorm_fwd(x, w, b)
    dx, dw, db = R.layernorm_bwd(x, dy, w, mean, rstd)

    def loss(x, w, b):
        return float((dy.double() * R.layernorm_fwd(x, w, b)[0].double()).sum())

    h = 0.02
    for which, grad in ((0, dx), (1, dw), (2, db)):
        args = [x, w, b]
        v = rand(g, *args[which].shape)
        f = []
        for k in (-2, -1, 1, 2):
            moved = list(args)
            moved[which] = args[which] + k * h * v
            f.append(loss(*moved))
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h)
        want = float((grad.double() * v.double()).sum())
        assert abs(fd - want) <= 1e-3 * float((grad.double() * v.double()).norm()) * 10


def test_other_stream_and_graph(R):
    g = gen(12)
    x, dy, w = rand(g, 64, 1024), rand(g, 64, 1024), rand(g, 1024)
    want_y, mean, rstd = R.layernorm_fwd(x, w)
    want = R.layernorm_bwd(x, dy, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, m, r = R.layernorm_fwd(x, w, stream=s)
    got = R.layernorm_bwd(x, dy, w, m, r, stream=s)
    s.synchronize()
    assert torch.equal(y, want_y) and all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, m2, r2 = R.layernorm_fwd(x, w)
        got2 = R.layernorm_bwd(x, dy, w, m2, r2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y2, want_y) and all(torch.equal(a, b) for a, b in zip(got2, want))
