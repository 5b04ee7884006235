"""GPU tests of the causal convolution where a thread walks a long run of tokens
(28 to 108 forward, 32 to 72 backward; small calls have runs of 4): windows that are
shifted many times, rings of loads that come round, runs that end in a sequence's
padding.  Bounds as in tests/ssm_reference.py: its sums over tokens count
64 + 64 additions a thread, a run has at most 128 tokens.
"""
import pytest
import torch

from tests.test_conv_gpu import BF16, F32, R, check, gen, rand  # noqa: F401 (R: fixture)

pytestmark = pytest.mark.gpu


# E a multiple of 4, even, odd: channels a thread 4 (backward in fp32 2), 1 (2), 1
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,E,W", [(1, 8191, 4096, 4), (2, 4001, 4098, 4), (3, 2701, 4097, 4), (40, 301, 1024, 3),
                                     (40, 301, 1030, 2), (40, 301, 1023, 4), (2, 4001, 2052, 2)])
def test_long_runs(R, dtype, B, N, E, W):
    g = gen(B * 100 + N * 7 + E + W)
    x, dy = rand(g, B, N, E, dtype=dtype), rand(g, B, N, E, dtype=dtype)
    w, b = rand(g, E, W, scale=0.5), rand(g, E, scale=0.1)
    state, ds = rand(g, B, W - 1, E, dtype=dtype), rand(g, B, W - 1, E, dtype=dtype)
    check(R, x, w, b, dy, state, ds)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,E,W", [(40, 301, 1024, 4), (40, 301, 1030, 3), (40, 301, 1023, 4), (4, 3001, 1028, 4)])
def test_padded_long_runs(R, dtype, B, N, E, W):
    """Lengths that end anywhere in a run, at its ends, and before the taps; NaN behind them."""
    g = gen(B + N + E)
    lengths = torch.randint(0, N + 1, (B,), generator=g, device="cuda")
    for i, n in enumerate((N, 0, 1, W - 2, 28, 29, 43, 44, 56, 88, N - 1)[:B - 1 if B < 11 else 11]):
        lengths[i] = n
    x, dy = rand(g, B, N, E, dtype=dtype), rand(g, B, N, E, dtype=dtype)
    behind = (torch.arange(N, device="cuda") >= lengths[:, None])[..., None]
    x, dy = x.masked_fill(behind, float("nan")), dy.masked_fill(behind, float("nan"))
    state, ds = rand(g, B, W - 1, E, dtype=dtype), rand(g, B, W - 1, E, dtype=dtype)
    w, b = rand(g, E, W), rand(g, E)
    y, _, dx, *rest = check(R, x, w, b, dy, state, ds, lengths.int())
    assert bool((y.masked_select(behind) == 0).all())
    same = R.causal_conv_bwd(x, w, b, dy, state_in=state, dstate_out=ds, lengths=lengths)
    assert torch.equal(same[0], dx) and all(torch.equal(p, q) for p, q in zip(same[1:], rest))
