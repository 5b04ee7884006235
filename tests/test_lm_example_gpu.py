"""The output head's operators together, as examples/distill_head.py runs them."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location(
        "distill_head", os.path.join(ROOT, "examples", "distill_head.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_head_learns_from_the_teacher(example):
    """Gradient descent on the framework's gradients: the loss never rises by
    more than 5% of itself and ends below half of where it began."""
    losses, _ = example.train(steps=20)
    assert all(b <= 1.05 * a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.5 * losses[0], losses


def test_scores_agree_with_64_bits(example):
    """The scores of the example's own logits, at token_logprobs' bound."""
    _, state = example.train(steps=3)
    logits, tokens, (logprob, entropy, top_lp, top_ids) = example.score(state)
    lp = torch.log_softmax(logits[:, :-1].double(), -1)
    for got, ref in ((logprob, lp.gather(-1, tokens[..., None])[..., 0]),
                     (entropy, -(lp.exp() * lp).sum(-1)), (top_lp, lp.topk(5, dim=-1).values)):
        assert bool(((got.double() - ref).abs() <= 1e-5 * (1 + ref.abs())).all())
    assert torch.equal(lp.gather(-1, top_ids), lp.topk(5, dim=-1).values)
