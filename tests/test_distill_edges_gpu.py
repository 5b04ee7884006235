"""GPU tests of the distillation loss where a teacher's probability is at the
bottom of fp32 and where the listed probabilities add up to more than 1, against
the formulas in 64 bits; the cross entropy that a list of one token is.
Tolerances: those of test_distill_gpu.py."""
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


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [0.5, 1.0])
def test_probabilities_at_the_bottom_of_fp32(R, T, dtype, tail):
    """Entries whose probability is denormal or nearly so (padding with a low
    log probability) for tokens that the student likes, a little or very much:
    the term is the student's q, not p times an e^(ln q - ln p) beyond fp32."""
    g = D.gen(31)
    low = torch.tensor([0.0, -60.0, -86.0, -88.0, -90.0, -95.0, -100.0, -103.0, -104.0, -120.0], device="cuda")
    x = torch.randn(11, 300, generator=g, device="cuda").to(dtype)
    ids = torch.randperm(300, generator=g, device="cuda")[:10].expand(11, 10).contiguous()
    for j in range(10):  # row j likes entry j with all but e^-20, row 10 all of them
        x[j, ids[j, j]] = 25.0
    x[10, ids[10]] = 12.0
    values = low if tail else low * T
    values = (values - (0.7 if tail else 0.0)).expand(11, 10).contiguous()
    ref = D.reference(x, ids, values, T, tail)
    loss, stats = R.distill_fwd(x, ids, values, temperature=T, tail=tail)
    assert bool(torch.isfinite(loss).all())
    D.check_loss(loss, ref[0], T)
    loss2, grad = R.distill_step(x, ids, values, temperature=T, tail=tail)
    assert torch.equal(loss2, loss)
    one = torch.ones(11, device="cuda")
    D.check_grad(grad, ref[1], ref[2], one, 160.0)
    D.check_grad(R.distill_bwd(x, ids, values, None, stats, temperature=T, tail=tail), ref[1], ref[2], one, 160.0)


def over_full(g, x, k, how):
    """(ids, values) of a teacher whose listed probabilities do not add up to
    one: log probabilities rounded to bf16 of nearly all of its mass, ones that
    were scaled by 1.5, and (k the whole vocabulary) by 0.5."""
    t = x.float() + torch.randn(x.shape, generator=g, device="cuda")
    v, ids = (2.0 * t).log_softmax(-1).topk(k, dim=-1)
    v = {"bf16": v.bfloat16().float(), "more": v + 0.4, "less": v - 0.7}[how]
    return ids.contiguous(), v.contiguous()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("V,k,how", [(130, 128, "bf16"), (31, 31, "bf16"), (3001, 100, "bf16"), (500, 100, "more"),
                                     (31, 31, "more"), (31, 31, "less"), (40003, 128, "more")])
def test_listed_probabilities_beyond_one(R, V, k, how, T, dtype):
    """The loss is the sum of p ln(p / q) all the same, and the gradient its
    derivative: T (P q_j - p_j) for the listed, P the sum of all p."""
    g = D.gen(V + k)
    x = (2.0 * torch.randn(6, V, generator=g, device="cuda")).to(dtype)
    ids, values = over_full(g, x, k, how)
    loss64, grad64, size, _ = D.reference(x, ids, values, T, True)
    listed = values.double().exp().sum(-1)
    total = torch.where((listed > 1) | (k == V), listed, 1.0)
    if how != "bf16":
        assert bool(((total - 1).abs() > 0.1).all())
    q = (x.double() / T).softmax(-1)
    grad64 = grad64 + T * (total - 1)[:, None] * q
    size = size * total.clamp(min=1.0)[:, None]
    loss, stats = R.distill_fwd(x, ids, values, temperature=T, tail=True)
    tol = T * T * 8e-6 + 1e-5 * loss64.abs()
    assert bool(((loss.double() - loss64).abs() <= tol).all())
    loss2, grad = R.distill_step(x, ids, values, temperature=T, tail=True)
    assert torch.equal(loss2, loss)
    one = torch.ones(6, device="cuda")
    D.check_grad(grad, grad64, size, one)
    D.check_grad(R.distill_bwd(x, ids, values, None, stats, temperature=T, tail=True), grad64, size, one)


@pytest.mark.parametrize("V,k,how", [(500, 100, "more"), (31, 31, "less")])
def test_gradient_against_differences_beyond_one(R, V, k, how):
    """Five-point differences of the loss (step 0.05: truncation below h^4 = 6e-6
    of a fifth derivative of the gradient's size, rounding of losses up to 4
    about 8e-6 / h = 2e-4 each) within 2e-3 of the gradient's size."""
    g = D.gen(40)
    x = 2.0 * torch.randn(3, V, generator=g, device="cuda")
    ids, values = over_full(g, x, k, how)
    _, grad = R.distill_step(x, ids, values, temperature=1.5, tail=True)
    h = 0.05
    for _ in range(3):
        v = torch.randn(3, V, generator=g, device="cuda")
        f = [R.distill_fwd(x + j * h * v, ids, values, temperature=1.5, tail=True)[0].double() for j in (-2, -1, 1, 2)]
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h)
        want = (grad.double() * v.double()).sum(-1)
        assert bool(((fd - want).abs() <= 2e-3 * grad.double().norm(dim=-1) + 4e-4).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_listed_token_is_cross_entropy(R, dtype):
    """Next-token cross entropy with ignored positions: loss, and the gradient
    of the mean over the others."""
    g = D.gen(41)
    x = (2.0 * torch.randn(3, 5, 5003, generator=g, device="cuda")).to(dtype)
    tokens = torch.randint(0, 5003, (3, 5), generator=g, device="cuda")
    tokens[0, 4] = tokens[2, 0] = -100
    there = tokens >= 0
    weight = torch.full((3, 5), 1.0 / float(there.sum()), device="cuda")
    loss, grad = R.distill_step(x, tokens[..., None], torch.zeros(3, 5, 1, device="cuda"), weight)
    lp = x.double().log_softmax(-1)
    D.check_loss(loss, torch.where(there, -lp.gather(-1, tokens.clamp(min=0)[..., None])[..., 0], 0.0), 1.0)
    one = torch.zeros_like(lp).scatter_(-1, tokens.clamp(min=0)[..., None], 1.0)
    D.check_grad(grad, (lp.exp() - one) * there[..., None], lp.exp() + one, weight)
    assert float(grad[~there].float().abs().max()) == 0
