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
