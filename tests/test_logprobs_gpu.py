"""GPU tests of token_logprobs against the definitions in 64 bits.

Tolerances, from fp32 arithmetic (u = 2^-24): a hardware exponential is good
to 2^-22 and its argument, at most 40 in size where it matters, to 40 u * 2;
so z has a relative error below 1e-5 / 2 and ln z an absolute one; a log
probability adds a few u of its size: 5e-6 (1 + |lp|).  The entropy's second
term is a mean of terms with the same relative error: 1e-5 (1 + H).
Ids are compared exactly (order by logit, then by the lower id).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits(g, *shape, dtype=torch.bfloat16, scale=3.0):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def reference(x, tokens, top, T):
    """Definitions in 64 bits; rows of finite values and -inf."""
    x64 = x.double()
    lp = torch.log_softmax(x64 / T, -1)
    dead = (x64 == -INF).all(-1)
    lp = torch.where(dead[..., None], -INF, lp)
    p = lp.exp()
    H = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    out = None
    if tokens is not None:
        out = lp.gather(-1, tokens.clamp(min=0)[..., None].long())[..., 0]
        out = torch.where(tokens < 0, 0.0, out)
    ids = torch.sort(x64 + 0.0, dim=-1, descending=True, stable=True).indices[..., :top]
    vals = lp.gather(-1, ids)
    ids = torch.where(x64.gather(-1, ids) == -INF, -1, ids)
    if top > x.shape[-1]:
        pad = top - x.shape[-1]
        ids = torch.nn.functional.pad(ids, (0, pad), value=-1)
        vals = torch.nn.functional.pad(vals, (0, pad), value=-INF)
    return out, H, vals, ids


def near(got, ref, tol):
    got = got.double()
    assert torch.equal(torch.isinf(got), torch.isinf(ref)) and not bool(torch.isnan(got).any())
    fin = torch.isfinite(ref)
    err = (got - ref)[fin].abs()
    lim = tol * (1 + ref[fin].abs())
    assert bool((err <= lim).all()), f"{float((err / lim).max()):.2f} times the tolerance"


def check(R, x, top, T=1.0, tokens=None):
    if tokens is None:
        tokens = torch.randint(0, x.shape[-1], x.shape[:-1], device="cuda")
    lp, H, tv, ti = R.token_logprobs(x, tokens, top=top, temperature=T)
    rlp, rH, rv, ri = reference(x, tokens, top, T)
    near(lp, rlp, 5e-6)
    near(H, rH, 1e-5)
    if top:
        assert torch.equal(ti, ri)
        near(tv, rv, 5e-6)
    else:
        assert tv is None and ti is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,top", [
    (1, 1, 1), (2, 1, 3), (3, 2, 1), (4, 7, 7), (5, 8, 3), (3, 9, 20), (6, 17, 5), (300, 256, 10),
    (7, 1000, 128), (3, 4095, 1), (2, 4097, 0), (5, 5003, 20), (9, 32768, 20), (2, 50001, 128),
    (1, 131072, 20), (8, 131072, 1), (200, 20000, 8), (1, 300000, 64), (700, 8192, 0)])
def test_sizes(R, dtype, rows, V, top):
    g = gen(rows * 31 + V)
    check(R, logits(g, rows, V, dtype=dtype), top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,top", [(1000, 20011, 5), (400, 9001, 100), (200, 40011, 40),
                                        (330, 2001, 33), (290, 20000, 2)])
def test_many_rows_with_masks_and_ties(R, dtype, rows, V, top):
    """Rows in several turns of the CTAs; among them rows with masked tokens,
    with the type's lowest value, masked throughout, and of few distinct values."""
    g = gen(rows + V)
    x = logits(g, rows, V, dtype=dtype)
    x[1::7] = torch.where(torch.rand(x[1::7].shape, generator=g, device="cuda") < 0.5, -INF, x[1::7].float()).to(dtype)
    x[2::7, V // 2:] = torch.finfo(dtype).min
    x[3::7] = -INF
    x[4::7] = x[4::7].round()
    x[5::7] = 1.5
    check(R, x, top, tokens=torch.randint(0, V // 2, (rows,), generator=g, device="cuda"))


@pytest.mark.parametrize("T", [0.01, 0.7, 3.0, 100.0])
def test_temperature(R, T):
    g = gen(2)
    check(R, logits(g, 5, 3001), 10, T)
    check(R, logits(g, 5, 3001, dtype=torch.float32), 10, T)


def test_strided_rows_and_int32_tokens(R):
    """logits[:, :-1] of a batch, a padded vocabulary, rows off the 16-byte
    boundary, the batch as the inner dimension."""
    g = gen(3)
    full = logits(g, 3, 9, 1003)
    for x in (full[:, :-1], full[..., :1000], full[..., 5:998], full.transpose(0, 1)[1:],
              logits(g, 2, 2, 3, 640, dtype=torch.float32)):
        check(R, x, 12, tokens=torch.randint(0, x.shape[-1], x.shape[:-1], device="cuda",
                                             dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [37, 4096, 50001])
def test_masks(R, dtype, V):
    """Most tokens masked; all but three; a mask of the type's lowest value;
    everything masked; a token that is masked; no token."""
    g = gen(V)
    x = logits(g, 8, V, dtype=dtype)
    keep = torch.rand(8, V, generator=g, device="cuda")
    x[0][keep[0] < 0.9] = -INF
    x[1][:] = -INF
    x[1][[1, V // 2, V - 1]] = torch.tensor([2.0, 2.0, 3.0], device="cuda").to(dtype)
    low = torch.finfo(dtype).min
    x[2][:] = low
    x[2][[0, V // 3]] = 1.0
    x[3] = -INF
    x[4][5] = -INF
    x[5] = low
    tokens = torch.randint(0, V, (8,), generator=g, device="cuda")
    tokens[0] = int(x[0].float().argmax())
    tokens[1], tokens[2], tokens[3], tokens[4], tokens[6] = 1, 1, 2, 5, -100
    check(R, x, 20, tokens=tokens)
    lp, H, _, ti = R.token_logprobs(x, tokens, top=20)
    assert float(lp[3]) == -INF and float(H[3]) == 0 and bool((ti[3] == -1).all())
    assert float(lp[4]) == -INF and float(lp[6]) == 0
    assert ti[1].tolist() == [V - 1, 1, V // 2] + [-1] * 17
    assert abs(float(H[5]) - math.log(V)) <= 1e-5 * (1 + math.log(V))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [1, 20, 128])
def test_ties_and_order(R, dtype, top):
    """Equal logits by the lower id: constant rows, two values, a few integer
    values, signed zeros, sorted rows, and large values that few threads of
    the kernel share (columns 4096 apart)."""
    g = gen(4)
    V = 40003
    x = torch.zeros(9, V, device="cuda")
    x[1] = -5.5
    x[2] = (torch.arange(V, device="cuda") % 3 == 1).float()
    x[3] = torch.randint(-4, 5, (V,), generator=g, device="cuda").float()
    x[4][::2] = -0.0
    x[5] = torch.linspace(8, -8, V, device="cuda")
    x[6] = torch.linspace(-8, 8, V, device="cuda")
    x[7][3::4096] = 5.0
    x[7][4::4096] = 6.0
    x[8] = torch.randn(V, generator=g, device="cuda")
    x[8][torch.arange(0, V, device="cuda") % 4096 < 16] += 30.0
    check(R, x.to(dtype), top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_large_values_in_few_threads(R, dtype):
    """More distinct values above the threads' bound than the kernel ranks at
    once: every 4096th group of 16 columns holds large ones."""
    g = gen(14)
    V = 1 << 20
    x = torch.randn(2, V, generator=g, device="cuda")
    cols = torch.arange(V, device="cuda") % 4096 < 16
    x[0][cols] = 20.0 + 10.0 * torch.rand(int(cols.sum()), generator=g, device="cuda")
    x[1][cols] = 20.0
    check(R, x.to(dtype), 128)


def test_nan_and_infinity(R):
    g = gen(5)
    x = logits(g, 5, 777, dtype=torch.float32)
    x[1, 700] = float("nan")
    x[3, 2] = INF
    tok = torch.tensor([1, 1, 1, 1, 776], device="cuda")
    lp, H, tv, ti = R.token_logprobs(x, tok, top=4)
    for r in (1, 3):
        assert math.isnan(lp[r]) and math.isnan(H[r])
        assert bool(torch.isnan(tv[r]).all()) and bool((ti[r] == -1).all())
    keep = [0, 2, 4]
    want = reference(x[keep], tok[keep], 4, 1.0)
    near(lp[keep], want[0], 5e-6)
    assert torch.equal(ti[keep], want[3])
    # a token past the vocabulary gives NaN, and reads nothing
    bad, _, _, _ = R.token_logprobs(x[:1], torch.tensor([777], device="cuda"))
    assert math.isnan(bad[0])


def test_large_and_extreme_levels(R):
    g = gen(6)
    x = logits(g, 4, 2050, dtype=torch.float32)
    x[0] += 1e6  # log probabilities keep the spacing of the logits themselves
    x[1] = torch.where(x[1] > 0, 3e38, -3e38)
    x[2] = 0.0
    x[2, 9] = 200.0
    tokens = x.argmax(-1)  # row 1's other tokens are beyond fp32's range
    check(R, x, 5, tokens=tokens)


def test_no_rows_and_no_tokens(R):
    x = torch.empty(0, 50, device="cuda")
    lp, H, tv, ti = R.token_logprobs(x, torch.empty(0, dtype=torch.int64, device="cuda"), top=3)
    assert lp.shape == (0,) and ti.shape == (0, 3)
    y = torch.randn(50, device="cuda")
    lp, H, tv, ti = R.token_logprobs(y, top=2)
    assert lp is None and H.shape == () and int(ti[0]) == int(y.argmax())


def test_long_row_offsets(R):
    """A row that starts past 2^31 elements."""
    V, rows = 65536, 32800
    x = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    x[-1, 123] = 4.0
    lp, H, tv, ti = R.token_logprobs(x[-2:], torch.tensor([0, 123], device="cuda"), top=2)
    view = torch.as_strided(x, (2, V), ((rows - 1) * V, 1))
    lp2, _, _, ti2 = R.token_logprobs(view, torch.tensor([0, 123], device="cuda"), top=2)
    assert torch.equal(lp, lp2) and ti2.tolist() == [[0, 1], [123, 0]] and torch.equal(ti, ti2)


def test_other_stream_and_graph(R):
    g = gen(7)
    x = logits(g, 16, 9001)
    tok = torch.randint(0, 9001, (16,), device="cuda")
    want = R.token_logprobs(x, tok, top=20)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = R.token_logprobs(x, tok, top=20, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = R.token_logprobs(x, tok, top=20)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
