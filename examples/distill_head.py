"""Distils a language model's output head from a teacher, step by step with
the library's own operators:

    hidden states of a RetNet block (retnet_block_fwd)
      -> final LayerNorm (layernorm_fwd) -> logits (gemm_bf16)
      -> loss and gradient against the teacher's top tokens (distill_step)
      -> gradients of the head (gemm_bf16) and of the LayerNorm (layernorm_bwd)
      -> an update of the head, the gains and the biases;

then scores the next tokens under the student (token_logprobs).  The teacher is
a head of its own on the same hidden states; its list, the 64 most probable
tokens with their log probabilities, comes from token_logprobs as well.
Weights are random, inputs synthetic.

    python examples/distill_head.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_recurrent_sequence_gb300 import retention as R  # noqa: E402
from linear_recurrent_sequence_gb300 import synth  # noqa: E402

B, N, D, H, DK, DV, FFN, VOCAB, TOP = 2, 256, 256, 2, 64, 128, 512, 2048, 64
TEMPERATURE = 2.0


def hidden_states(seed):
    """The output of one RetNet block on random token embeddings, [B, N, D]."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def w(*shape, scale=0.05):
        return (scale * torch.randn(*shape, generator=g, device="cuda")).bfloat16()

    ln = [torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")]
    return R.retnet_block_fwd(w(B, N, D, scale=1.0), *ln, w(D, H * DK), w(D, H * DK), w(D, H * DV),
                              w(D, H * DV), w(H * DV, D), *ln, w(D, FFN), w(FFN, D), H=H, d_k=DK,
                              d_v=DV, gamma=synth.head_gammas(H), norm_flags=R.NORM_ALL)


def train(steps=30, lr=20.0, seed=1):
    """The mean loss before each step, and the last gradients' sizes."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    h = hidden_states(seed)
    rows = B * N
    # the teacher's list for every position
    teacher = (0.3 * torch.randn(D, VOCAB, generator=g, device="cuda")).bfloat16()
    x, _, _ = R.layernorm_fwd(h)
    logits = R.gemm_bf16(x.view(rows, D), teacher).view(B, N, VOCAB)
    _, _, values, ids = R.token_logprobs(logits, top=TOP, temperature=TEMPERATURE)

    head = torch.zeros(D, VOCAB, device="cuda")  # fp32 master weights
    gain, bias = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
    weight = torch.full((B, N), 1.0 / rows, device="cuda")
    weight[:, -1] = 0.0  # the last position has no next token: no gradient
    losses = []
    for _ in range(steps):
        w16 = head.bfloat16()
        x, mean, rstd = R.layernorm_fwd(h, gain, bias)
        x2 = x.view(rows, D)
        student = R.gemm_bf16(x2, w16).view(B, N, VOCAB)
        # the gradient takes the logits' place
        loss, d = R.distill_step(student, ids, values, weight, temperature=TEMPERATURE, tail=True,
                                 dstudent=student)
        losses.append(float((loss * weight).sum()))
        d = d.view(rows, VOCAB)
        dhead = R.gemm_bf16(x2.t().contiguous(), d)
        dx = R.gemm_bf16(d, w16.t().contiguous()).view(B, N, D)
        _, dgain, dbias = R.layernorm_bwd(h, dx, gain, mean, rstd)
        head -= lr * dhead.float()
        gain -= 0.1 * lr * dgain
        bias -= 0.1 * lr * dbias
    return losses, (h, head, gain, bias)


def score(state, seed=7):
    """The logits, random next tokens of each position but the last, and their
    scores: log probability, entropy and the five most probable tokens."""
    h, head, gain, bias = state
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x, _, _ = R.layernorm_fwd(h, gain, bias)
    logits = R.gemm_bf16(x.view(B * N, D), head.bfloat16()).view(B, N, VOCAB)
    tokens = torch.randint(0, VOCAB, (B, N - 1), generator=g, device="cuda")
    return logits, tokens, R.token_logprobs(logits[:, :-1], tokens, top=5)


def main():
    losses, state = train()
    for i in range(0, len(losses), 5):
        print(f"step {i:3d}  loss {losses[i]:.4f}")
    print(f"last      loss {losses[-1]:.4f}")
    _, tokens, (logprob, entropy, top_lp, top_ids) = score(state)
    print(f"mean log probability of random next tokens {float(logprob.mean()):.3f}, "
          f"mean entropy {float(entropy.mean()):.3f}")
    print("first position:", ", ".join(f"{int(i)} ({float(p):.2f})"
                                       for i, p in zip(top_ids[0, 0], top_lp[0, 0])))


if __name__ == "__main__":
    main()
