"""GPU tests of the RMS norm's e4m3 output at the sizes where its kernels change
their way: rows that one warp reads again, several rows a CTA one after another.

Bounds as in tests/test_rmsnorm_gpu.py: y within units(d) of itself, the scale
4 u more, an e4m3 value off by half a step (2^-4 of itself, 2^-10 below the normal
range) and the error of its quotient, units(d) and 10 u.
"""
import pytest
import torch

from tests.test_rmsnorm_gpu import BF16, F32, R, U, gen, kept, normed, rand, units  # noqa: F401 (R: fixture)

pytestmark = pytest.mark.gpu


def check_quant(q, scales, h, w, group, eps=1e-5):
    """q and scales of the kept rows h [rows, d]."""
    d = h.shape[-1]
    size = min(group or d, d)
    y = normed(h, w, eps)[1]
    pad = -d % size
    blocks = torch.nn.functional.pad(y, (0, pad)).unflatten(-1, (-1, size))
    values = torch.nn.functional.pad(q.float(), (0, pad)).unflatten(-1, (-1, size)).double()
    want, k = blocks.abs().amax(-1) / 448.0, units(d)
    assert scales.shape == want.shape and bool(((scales.double() - want).abs() <= (k + 4 * U) * want).all())
    s = scales.double()[..., None]
    exact = torch.where(s > 0, blocks / s.clamp(min=1e-300), 0.0)
    tol = (exact.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) + exact.abs() * (k + 10 * U)
    assert bool(((values - exact).abs() <= tol).all())
    assert bool(((values.abs().amax(-1) == 448.0) | (s[..., 0] == 0)).all())


@pytest.mark.parametrize("dtype,d", [(BF16, 257), (BF16, 300), (BF16, 509), (F32, 301), (F32, 511)])
@pytest.mark.parametrize("group", [16, 40, 0])
def test_many_rows_that_one_warp_reads_again(R, dtype, d, group):
    """Rows of 257 to 512 values off the 16-byte boundary, too many for all at once:
    the sum that one lane keeps is what another lane scales."""
    rows = 9001
    g = gen(d + group)
    x, r, w = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    for res in (r, None):
        q, scales, h = R.rmsnorm_quant(x, w, residual=res, group=group)
        assert torch.equal(h, kept(x, res))
        check_quant(q, scales, h, w, group)
    a, b = x.clone(), r.clone()  # kept in place of either
    q2, s2, h2 = R.rmsnorm_quant(a, w, residual=b, group=group, residual_out=a)
    q3, s3, _ = R.rmsnorm_quant(x, w, residual=r, group=group)
    assert h2 is a and torch.equal(q2.view(torch.uint8), q3.view(torch.uint8)) and torch.equal(s2, s3)


# rows by one of the kernels each: a lane's group, a warp's, half a warp's, the row's, read again
SHAPES = [(BF16, 40, 64, 8), (BF16, 40, 512, 128), (F32, 40, 512, 128), (BF16, 40, 4096, 256), (F32, 7, 1000, 40),
          (BF16, 9, 130, 0), (F32, 9001, 301, 16), (BF16, 3, 20001, 128), (BF16, 2, 40000, 2048)]


@pytest.mark.parametrize("dtype,rows,d,group", SHAPES)
def test_groups_with_nan(R, dtype, rows, d, group):
    """The scale of a group that has a NaN is NaN, and so are its values; a NaN gain
    stays in its group, a NaN in the row is in all of them."""
    g = gen(rows + d)
    x, w = rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    size = min(group or d, d)
    want_q, want_s, _ = R.rmsnorm_quant(x, w, group=group)
    bad = x.clone()
    bad[1, d // 2] = float("nan")
    q, s, _ = R.rmsnorm_quant(bad, w, group=group)
    rest = [i for i in range(rows) if i != 1]
    assert bool(torch.isnan(s[1]).all()) and bool(torch.isnan(q[1].float()).all())
    assert torch.equal(q.view(torch.uint8)[rest], want_q.view(torch.uint8)[rest]) and torch.equal(s[rest], want_s[rest])
    for nan in (float("nan"), -float("nan")):
        w2 = w.clone()
        w2[d // 2] = nan
        q, s, _ = R.rmsnorm_quant(x, w2, group=group)
        hit = (torch.arange(d, device="cuda") // size) == d // 2 // size
        assert bool(torch.isnan(s[:, d // 2 // size]).all()) and bool(torch.isnan(q.float()[:, hit]).all())
        assert torch.equal(q.view(torch.uint8)[:, ~hit], want_q.view(torch.uint8)[:, ~hit])
        keep = torch.arange(s.shape[-1], device="cuda") != d // 2 // size
        assert torch.equal(s[:, keep], want_s[:, keep])


@pytest.mark.parametrize("dtype,rows,d,group", SHAPES)
def test_groups_with_infinity(R, dtype, rows, d, group):
    """An infinite value makes its group's scale infinite: y / scale is NaN for
    itself and 0 for the group's finite values."""
    g = gen(rows + d)
    x, w = rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    x[:, d // 2] = 1.0
    size = min(group or d, d)
    want_q, want_s, _ = R.rmsnorm_quant(x, w, group=group)
    for inf in (float("inf"), -float("inf")):
        w2 = w.clone()
        w2[d // 2] = inf
        q, s, _ = R.rmsnorm_quant(x, w2, group=group)
        hit = (torch.arange(d, device="cuda") // size) == d // 2 // size
        assert bool((s[:, d // 2 // size] == float("inf")).all()) and bool(torch.isnan(q.float()[:, d // 2]).all())
        zeros = hit.clone()
        zeros[d // 2] = False
        assert bool((q.float()[:, zeros] == 0).all())
        assert torch.equal(q.view(torch.uint8)[:, ~hit], want_q.view(torch.uint8)[:, ~hit])
        keep = torch.arange(s.shape[-1], device="cuda") != d // 2 // size
        assert torch.equal(s[:, keep], want_s[:, keep])
    # an infinite value in the row: its norm is infinite, rstd 0, and inf x 0 is NaN
    bad = x.clone()
    bad[1, d // 2] = float("inf")
    q, s, _ = R.rmsnorm_quant(bad, w, group=group)
    assert bool(torch.isnan(s[1, d // 2 // size])) and bool((s[1][torch.arange(s.shape[-1], device="cuda") != d // 2 // size] == 0).all())
    assert bool((q.float()[1, ~hit] == 0).all()) and bool(torch.isnan(q.float()[1, hit]).all())


@pytest.mark.parametrize("rows,d,group", [(20000, 256, 8), (4096, 4096, 128), (500, 16384, 0), (1000, 1001, 40)])
def test_quotients_are_rounded_once(R, rows, d, group):
    """In fp32 the norm's own output holds y as the e4m3 form has it before the
    division: the scales are max |y| / 448 and the values y / scale, both rounded as
    fp32 divides, then to the nearest e4m3 value, bit for bit.  (Among 10^7 quotients
    some lie within half a unit of a border between two e4m3 values.)  The rows are
    ones that both forms take through one kernel: rows that are read again have their
    mean rounded differently."""
    g = gen(rows)
    x, w = rand(g, rows, d), 1.0 + rand(g, d, scale=0.1)
    y, _, _ = R.rmsnorm_fwd(x, w)
    q, s, _ = R.rmsnorm_quant(x, w, group=group)
    size = group or d
    blocks = torch.nn.functional.pad(y, (0, -d % size)).unflatten(-1, (-1, size))
    # (a tensor: torch multiplies by the reciprocal of a number)
    assert torch.equal(s, blocks.abs().amax(-1) / torch.full_like(s, 448.0))
    want = (blocks / s[..., None]).flatten(-2)[:, :d].to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


# more rows than run at once, no multiple of a CTA's: short rows of a part of a warp, of
# a warp, of several; groups of a lane, half a warp, a warp, the row
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,d,group", [(20011, 64, 0), (20011, 100, 8), (5001, 512, 128), (3001, 768, 8), (1501, 4096, 128),
                                          (1501, 4096, 256), (1501, 4096, 0), (701, 16384, 128), (4001, 1000, 40)])
def test_more_rows_than_at_once(R, dtype, rows, d, group):
    g = gen(rows + d + group)
    x, r, w = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype), 1.0 + rand(g, d, scale=0.1)
    x *= 0.01 + torch.rand(rows, 1, generator=g, device="cuda").to(dtype)  # (each row has its own scales)
    for res in (r, None):
        q, scales, h = R.rmsnorm_quant(x, w, residual=res, group=group)
        assert torch.equal(h, kept(x, res))
        check_quant(q, scales, h, w, group)
        again = R.rmsnorm_quant(x, w, residual=res, group=group)
        assert torch.equal(q.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(scales, again[1])
