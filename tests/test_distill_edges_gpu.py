"""GPU tests of the distillation loss where a teacher's probability is at the
bottom of fp32, against the formulas in 64 bits.  Tolerances: those of
test_distill_gpu.py."""
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
