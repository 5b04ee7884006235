"""GPU tests of the LayerNorm's and the distillation's gradients against
five-point differences of their forward passes, at the bounds that rounding and
truncation give.

LayerNorm, sum(dy y) over 910 values with a step h = 0.02: truncation h^4 / 30 of
the fifth derivative, 5e-9 times 5! of the gradient's size; rounding of y by 3 u
(u = 2^-24) each, weighted 18 / 12, at most 4.5 u sum|dy y| / h = 730 * 1.4e-5 =
1e-2, where the sizes below are 20 and more: within 1e-3 of them.

Distillation, losses up to 6 with an error of 2e-6 (5 u of that), a
step of 0.05: rounding 1.5 * 2e-6 / h = 6e-5; truncation 2e-7 times 5! of the
gradient's size, which is far below 1e-3 of it.
"""
import pytest
import torch

from tests import test_distill_gpu as D

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


def five_points(f, h):
    a, b, c, d = (f(k * h) for k in (-2, -1, 1, 2))
    return (a - 8 * b + 8 * c - d) / (12 * h)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("which", range(3))
def test_layernorm(R, which, seed):
    g = D.gen(60 + seed)
    args = [D.randn(g, 7, 130), D.randn(g, 130), D.randn(g, 130)]
    dy = D.randn(g, 7, 130)
    _, mean, rstd = R.layernorm_fwd(*args)
    grad = R.layernorm_bwd(args[0], dy, args[1], mean, rstd)[which].double()
    v = D.randn(g, *args[which].shape)

    def at(step):
        moved = list(args)
        moved[which] = args[which] + step * v
        return float((dy.double() * R.layernorm_fwd(*moved)[0].double()).sum())

    size = float((grad * v.double()).norm())
    assert size >= 10
    assert abs(five_points(at, 0.02) - float((grad * v.double()).sum())) <= 1e-3 * size


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("tail", [False, True])
def test_distillation(R, tail, seed):
    g = D.gen(70 + seed)
    x = 2.0 * D.randn(g, 3, 1001)
    ids, values = D.teacher_of(g, x, 20, 1.5, tail)
    loss, grad = R.distill_step(x, ids, values, temperature=1.5, tail=tail)
    assert float(loss.max()) <= 6
    v = D.randn(g, 3, 1001)
    fd = five_points(lambda step: R.distill_fwd(x + step * v, ids, values, temperature=1.5, tail=tail)[0].double(), 0.05)
    want = (grad.double() * v.double()).sum(-1)
    assert bool(((fd - want).abs() <= 1e-3 * grad.double().norm(dim=-1) + 6e-5).all())
