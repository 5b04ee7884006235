"""GPU tests of the logits operators at levels where a logit times
log2(e) / T is far beyond the digits of fp32: finite mask constants, low
temperatures, rows, slices and warps that hold nothing else.

Tolerances: those of test_logprobs_gpu.py and test_distill_gpu.py, whose
derivations know differences from the row's maximum alone: such a difference is
rounded once whatever the level is.  Of the logits' spread only what is above
e^-104, fp32's smallest number, counts: at most 104 / ln 2 = 150 in the exponent
of 2, so the gradients are held to the bound of a spread of 160.
"""
import pytest
import torch

from tests import test_distill_gpu as D
from tests import test_logprobs_gpu as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


def rows_at(g, c, V, dtype):
    """Rows around the level c: nothing else; normal logits after and before
    a stretch of it; all but three tokens; all but the first ones; several
    such levels in any order, normal logits among them; neighbours of c."""
    x = (3.0 * torch.randn(7, V, generator=g, device="cuda")).to(dtype)
    x[0] = c
    x[1, :V // 2] = c
    x[2, V // 2:] = c
    keep = x[3, [0, V // 3, V - 1]].clone()
    x[3] = c
    x[3, [0, V // 3, V - 1]] = keep
    x[4, min(8, V - 1):] = c
    some = torch.tensor([c, c / 7, 3 * c, 1.001 * c, -4e6, -3e6, 1.0], device="cuda").to(dtype)
    pick = torch.randint(0, 7, (V,), generator=g, device="cuda")
    x[5] = torch.where(pick == 6, x[5], some[pick])
    near = torch.tensor([1.0, 1.01, 1.02, 1.05], device="cuda") * c
    x[6] = near.to(dtype)[torch.randint(0, 4, (V,), generator=g, device="cuda")]
    return x


def reference(x, ids, values, T, tail):
    """test_distill_gpu.reference with its softmaxes relative to their own
    maxima, since at these levels 64 bits lose ln z too (the sum of 1e20 and ln z
    is 1e20): the row's by moving the logits, which changes neither loss nor
    gradient (the statistics are moved back), and the rest bucket's by
    torch.softmax."""
    top = x.double().amax(-1, keepdim=True)
    loss, grad, size, stats = D.reference(x.double() - top, ids, values, T, tail)
    if tail:
        rest = (1 - values.double().exp().sum(-1, keepdim=True)).clamp(min=0)
        s = (x.double() / T).scatter(-1, ids, -L.INF)
        lost = rest * (((x.double() - top) / T - stats[..., 1:]).exp()).masked_fill(s == -L.INF, 0.0)
        moved = rest * s.softmax(-1)
        grad, size = grad + T * (lost - moved), size + T * (moved - lost)
    return loss, grad, size, stats + top / T


LEVELS = [-3e6, -1e9, -1e10, -1e20, -1e30, 1e10]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0.1, 1.0, 2.0])
@pytest.mark.parametrize("c", LEVELS)
def test_log_probabilities(R, c, T, dtype):
    g = L.gen(17)
    for V in (37, 5003, 131075):
        L.check(R, rows_at(g, c, V, dtype), 20, T)
    # single CTAs a row
    L.check(R, rows_at(g, c, 9001, dtype).repeat(100, 1), 0, T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1e-3, 1e-6, 1e-9])
def test_log_probabilities_at_low_temperatures(R, T, dtype):
    g = L.gen(18)
    x = L.logits(g, 6, 20011, dtype=dtype)
    x[1, 5:] = -1e9
    x[2] = 7.0
    L.check(R, x, 12, T)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0.1, 1.0, 2.0])
@pytest.mark.parametrize("c", LEVELS)
def test_distillation(R, c, T, dtype, tail):
    """Loss, statistics and the gradient of the same call.  Listed: random
    tokens and those that carry a row's normal logits."""
    g = L.gen(19)
    for V, k in ((37, 5), (5003, 20), (70001, 64)):
        x = rows_at(g, c, V, dtype)
        ids = torch.rand(7, V, generator=g, device="cuda")
        ids[:, [0, V // 3, V - 1]] += 1.0
        ids = ids.topk(k, dim=-1).indices
        values = torch.log_softmax(torch.randn(7, k + 1, generator=g, device="cuda"), -1)[:, :k].contiguous()
        loss, grad, size, stats = reference(x, ids, values, T, tail)
        got, got_stats = R.distill_fwd(x, ids, values, temperature=T, tail=tail)
        D.check_loss(got, loss, T)
        assert bool(((got_stats.double() - stats).abs() <= 4e-6 + 4e-7 * stats.abs()).all())
        got2, got_grad = R.distill_step(x, ids, values, temperature=T, tail=tail)
        assert torch.equal(got2, got)
        D.check_grad(got_grad, grad, size, torch.ones(7, device="cuda"), 160.0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0.1, 1.0, 2.0])
@pytest.mark.parametrize("c", LEVELS)
def test_gradient_from_saved_statistics(R, c, T, dtype, tail):
    """The gradient from the forward's statistics, an fp32 number of the size
    of the level: the probabilities have to keep their digits.  Over the
    logits too, and with rows of weight 0 among them."""
    g = L.gen(20)
    for V, k in ((37, 5), (5003, 20), (70001, 64)):
        x = rows_at(g, c, V, dtype)
        ids = torch.rand(7, V, generator=g, device="cuda")
        ids[:, [0, V // 3, V - 1]] += 1.0
        ids = ids.topk(k, dim=-1).indices
        values = torch.log_softmax(torch.randn(7, k + 1, generator=g, device="cuda"), -1)[:, :k].contiguous()
        weight = torch.rand(7, generator=g, device="cuda")
        weight[2] = 0.0
        _, grad, size, _ = reference(x, ids, values, T, tail)
        _, stats = R.distill_fwd(x, ids, values, temperature=T, tail=tail)
        got = R.distill_bwd(x, ids, values, weight, stats, temperature=T, tail=tail)
        D.check_grad(got, grad, size, weight, 160.0)
        over = x.clone()
        R.distill_bwd(over, ids, values, weight, stats, temperature=T, tail=tail, dstudent=over)
        D.check_grad(over, grad, size, weight, 160.0)


def test_statistics_beyond_fp32(R):
    """Levels that x / T takes out of fp32's range: q is uniform all the same."""
    for c in (3e38, -3e38):
        x = torch.full((2, 4099), c, device="cuda")
        ids = torch.tensor([[3, 700], [4098, -1]], device="cuda")
        values = torch.log(torch.tensor([[0.5, 0.25], [0.5, 0.25]], device="cuda"))
        for tail in (False, True):
            _, stats = R.distill_fwd(x, ids, values, temperature=0.5, tail=tail)
            got = R.distill_bwd(x, ids, values, None, stats, temperature=0.5, tail=tail)
            want = D.reference(torch.zeros_like(x), ids, values, 0.5, tail)
            D.check_grad(got, want[1], want[2], torch.ones(2, device="cuda"))


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_of_rows_at_several_levels(R, tail):
    """Many rows a CTA, ordinary and far ones in turn, rows without a teacher
    and of NaN among them."""
    g = L.gen(21)
    x = (2.0 * torch.randn(1400, 3001, generator=g, device="cuda"))
    x[1::3] += 5e4
    x[2::9] = -1e9
    x[5] = float("nan")
    x[8] = -L.INF
    ids = torch.rand(1400, 3001, generator=g, device="cuda").topk(10, dim=-1).indices
    values = torch.log_softmax(torch.randn(1400, 11, generator=g, device="cuda"), -1)[:, :10].contiguous()
    ids[4] = -1
    _, stats = R.distill_fwd(x, ids, values, tail=tail)
    got = R.distill_bwd(x, ids, values, None, stats, tail=tail)
    _, step = R.distill_step(x, ids, values, tail=tail)
    assert bool(torch.isnan(got[5]).all()) and float(got[8].abs().max()) == 0
    if not tail:
        assert float(got[4].abs().max()) == 0
    rows = [r for r in range(1400) if r not in (4, 5, 8)]
    _, grad, size, _ = D.reference(x[rows], ids[rows], values[rows], 1.0, tail)
    D.check_grad(got[rows], grad, size, torch.ones(len(rows), device="cuda"), 256.0)
    D.check_grad(step[rows], grad, size, torch.ones(len(rows), device="cuda"), 256.0)
