"""GPU tests of the selective scan where its kernels change with the size: steps of
so many sequences that a CTA walks over them several at a time, and gradients whose
partial sums over chunks are wide and many.  Bounds as in tests/ssm_reference.py."""
import pytest
import torch

from tests import test_scan_gpu as base
from tests.test_scan_gpu import BF16, F32, R, check_bwd, gen, problem, rand, ref, want  # noqa: F401 (R: fixture)

pytestmark = pytest.mark.gpu

# 1, 2, 4, 8 and 16 lanes a channel; sequences that are no multiple of the four (two,
# one) of a turn; several turns a CTA; S off the multiples of 4; groups
MANY = [(600, 2048, 4, 1), (1000, 1500, 3, 1), (259, 4099, 7, 1), (513, 2048, 8, 2), (130, 8192, 16, 1), (131, 4098, 13, 3),
        (66, 4096, 32, 1), (67, 4000, 17, 4), (41, 2048, 64, 1), (45, 2050, 33, 2)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,E,S,G", MANY)
def test_step(R, dtype, B, E, S, G):
    base.test_step(R, dtype, B, E, S, G)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,E,S,G", [(130, 8192, 16, 1), (259, 4100, 8, 2), (66, 4096, 32, 1)])
def test_step_on_slices(R, dtype, B, E, S, G):
    """Rows of wider buffers, B and C one value off the vectors' boundary, no gate,
    skip or bias, steps as they are: the values of contiguous tensors' call."""
    args, kw = problem(B, B, 1, E, S, G, dtype, gate=False, skip=False, bias=False)
    args[1] = args[1].abs() * 0.05
    w = want(args, dict(kw, softplus=False))
    wide = lambda t, before: torch.cat([t.new_full((B, before), 7.0), t.reshape(B, -1), t.new_full((B, 5), 7.0)], 1)[:, before:-5]
    x, dt = (wide(args[i][:, 0], 3) for i in (0, 1))
    Bm, Cm = (wide(args[i][:, 0], 1).unflatten(1, (G, S)) for i in (3, 4))
    buf = torch.full((B, E + 3), 7.0, dtype=dtype, device="cuda")
    h = kw["h_in"].clone()
    y = R.selective_scan_step(x, dt, args[2], Bm, Cm, h, softplus=False, out=buf[:, 1:E + 1])
    ref.check("y", y[:, None], w["y"])
    ref.check("h", h, w["h"])
    assert bool((buf[:, 0] == 7).all()) and bool((buf[:, E + 1:] == 7).all())


# column sums of 16384 (81920) and E columns in one launch: 132 parts and few
@pytest.mark.parametrize("dtype,B,N,E,S,G", [(BF16, 2, 2100, 1024, 16, 1), (F32, 3, 1430, 1024, 16, 2), (BF16, 2, 70, 5120, 16, 1),
                                             (F32, 1, 45, 2052, 8, 1)])
def test_wide_sums_over_chunks(R, dtype, B, N, E, S, G):
    args, kw = problem(B + N, B, N, E, S, G, dtype)
    g = gen(N)
    check_bwd(R, args, kw, rand(g, B, N, E, dtype=dtype), rand(g, B, E, S))
