"""GPU tests of the distillation loss and its gradient against the formulas in
64 bits.

Tolerances, from fp32 arithmetic (u = 2^-24): ln p, ln q and their difference
d carry an absolute error of at most e = 4e-6 (logits of size up to 40 here: a
few u of it each).  A loss term p (d - 1 + e^-d) then moves by p |1 - e^-d| e,
at most (p + q) e over all terms: |error| <= T^2 (2 e + 1e-5 L / T^2).  q and p
have a relative error of e, so a gradient value is within
w T (p + q + q') 1e-5 with q' = p_rest q / q_rest, plus half an ulp of a bf16
result.
"""
import math

import pytest
import torch

from tests.helpers import bf16_half_ulp

pytestmark = pytest.mark.gpu
INF = math.inf


def half_ulp(x):
    return torch.from_numpy(bf16_half_ulp(x.cpu().numpy())).to(x.device)


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


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def teacher_of(g, student, k, T, tail):
    """A teacher's list: the k largest of the student's logits with noise."""
    t = student.float() + randn(g, *student.shape)
    vals, ids = t.topk(k, dim=-1)
    if tail:
        vals = vals / T - torch.logsumexp(t / T, -1, keepdim=True)
    return ids.contiguous(), vals.contiguous()


def reference(student, ids, values, T, tail):
    """(loss, gradient without the weight, its scale, stats) in 64 bits, one
    row at a time; ids of a row distinct or negative."""
    V = student.shape[-1]
    x, idf, vf = student.double().reshape(-1, V), ids.reshape(-1, ids.shape[-1]), \
        values.double().reshape(-1, ids.shape[-1])
    losses, grads, sizes, stats = [], [], [], []
    for r in range(x.shape[0]):
        there = idf[r] >= 0
        k = idf[r][there].long()
        s = x[r] / T
        lse = torch.logsumexp(s, 0)
        q = (s - lse).exp()
        if tail:
            p = vf[r][there].exp()
            rest = (1 - p.sum()).clamp(min=0) * (k.numel() < V)
        else:
            p = torch.softmax(vf[r][there] / T, 0)
            rest = torch.zeros((), dtype=torch.float64, device=x.device)
        others = torch.ones(V, dtype=torch.bool, device=x.device)
        others[k] = False
        lse_rest = torch.logsumexp(s[others], 0) if bool(others.any()) else torch.tensor(-INF, dtype=torch.float64, device=x.device)
        loss = (torch.special.xlogy(p, p) - torch.where(p > 0, p * (s[k] - lse), 0.0)).sum()
        if float(rest) > 0:
            loss = loss + rest * (rest.log() - (lse_rest - lse))
        moved = rest * torch.where(others, (s - lse_rest).exp(), 0.0) if float(rest) > 0 else torch.zeros_like(q)
        dense = torch.zeros_like(q).index_add_(0, k, p)
        losses.append(T * T * loss)
        grads.append(T * (q - dense - moved))
        sizes.append(T * (q + dense + moved))
        stats.append(torch.stack([lse, lse_rest]))
    lead = student.shape[:-1]
    return (torch.stack(losses).reshape(lead), torch.stack(grads).reshape(student.shape),
            torch.stack(sizes).reshape(student.shape), torch.stack(stats).reshape(*lead, 2))


def check_loss(got, ref, T):
    tol = T * T * 8e-6 + 1e-5 * ref
    assert bool(((got.double() - ref).abs() <= tol).all()), \
        f"{float(((got.double() - ref).abs() / tol).max()):.2f} times the tolerance"


def check_grad(got, ref, size, w, spread=40.0):
    """e grows with the spread of the logits where that is above 40."""
    w = w.double()[..., None]
    tol = 1e-5 * spread / 40.0 * size * w.abs() + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol + half_ulp(ref * w)
    err = (got.double() - ref * w).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.2f} times the tolerance"


def check(R, student, ids, values, T=1.0, tail=False, weight=None, spread=40.0):
    ref = reference(student, ids, values, T, tail)
    w = torch.ones(student.shape[:-1], device="cuda") if weight is None else weight
    loss, stats = R.distill_fwd(student, ids, values, temperature=T, tail=tail)
    check_loss(loss, ref[0], T)
    fin = torch.isfinite(ref[3])
    assert torch.equal(torch.isfinite(stats), fin)
    assert bool(((stats.double() - ref[3])[fin].abs() <= 4e-6 + 4e-7 * ref[3][fin].abs()).all())
    grad = R.distill_bwd(student, ids, values, weight, stats, temperature=T, tail=tail)
    assert grad.dtype == student.dtype and grad.shape == student.shape
    check_grad(grad, ref[1], ref[2], w, spread)
    loss2, grad2 = R.distill_step(student, ids, values, weight, temperature=T, tail=tail)
    assert torch.equal(loss2, loss)
    check_grad(grad2, ref[1], ref[2], w, spread)
    return loss, stats, grad, grad2


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,k", [
    (1, 1, 1), (2, 2, 1), (3, 3, 3), (4, 9, 2), (5, 31, 31), (3, 130, 128), (7, 1000, 16),
    (5, 4097, 64), (2, 5003, 1), (9, 32768, 20), (3, 50001, 128), (170, 20011, 5),
    (2, 131072, 64), (1, 262147, 7)])
def test_sizes(R, dtype, tail, rows, V, k):
    g = gen(rows * 37 + V)
    student = (2.0 * randn(g, rows, V)).to(dtype)
    ids, values = teacher_of(g, student, k, 2.0, tail)
    weight = torch.rand(rows, generator=g, device="cuda") / rows
    check(R, student, ids, values, 2.0, tail, weight)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [0.5, 1.0, 4.0])
def test_strided_rows_and_int32_ids(R, T, tail):
    g = gen(2)
    full = (2.0 * randn(g, 3, 6, 1203)).bfloat16()
    for x in (full[:, :-1], full[..., :1200], full[..., 5:1000], full.transpose(0, 1),
              2.0 * randn(g, 2, 4, 640)):
        ids, values = teacher_of(g, x, 10, T, tail)
        check(R, x, ids.int(), values, T, tail)
    # a gradient inside a wider buffer of another alignment
    buf = torch.full((3, 6, 1300), 7.0, dtype=torch.bfloat16, device="cuda")
    ids, values = teacher_of(g, full, 10, T, tail)
    want = R.distill_step(full, ids, values, temperature=T, tail=tail)[1]
    R.distill_step(full, ids, values, temperature=T, tail=tail, dstudent=buf[..., 3:1206])
    assert torch.equal(buf[..., 3:1206], want)
    assert bool((buf[..., :3] == 7).all()) and bool((buf[..., 1206:] == 7).all())


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 4104), (torch.float32, 5003)])
@pytest.mark.parametrize("tail", [False, True])
def test_in_place(R, dtype, V, tail):
    g = gen(3)
    x = (2.0 * randn(g, 5, V)).to(dtype)
    ids, values = teacher_of(g, x, 30, 1.0, tail)
    loss, stats, grad, grad2 = check(R, x, ids, values, 1.0, tail)
    a, b = x.clone(), x.clone()
    assert torch.equal(R.distill_bwd(a, ids, values, None, stats, tail=tail, dstudent=a), grad)
    got = R.distill_step(b, ids, values, tail=tail, dstudent=b)
    assert torch.equal(got[0], loss) and torch.equal(b, grad2)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 70001), (torch.float32, 70001), (torch.bfloat16, 131080),
                                     (torch.float32, 300007)])
def test_repeated_ids_and_in_place_in_large_vocabularies(R, dtype, V, tail):
    """Entries of one token far apart in the list (the first counts, the same
    bits as without the others), at both ends of the row and between, and
    gradients over the logits where several CTAs share a row."""
    g = gen(V)
    x = (2.0 * randn(g, 2, V + 3)).to(dtype)[:, 3:]
    ids, values = teacher_of(g, x, 100, 1.0, tail)
    ids[0, :4] = torch.tensor([V - 1, 0, V // 2, V // 2 + 1], device="cuda")
    for r in range(2):  # distinct to begin with
        seen = set()
        for j, i in enumerate(ids[r].tolist()):
            if i in seen:
                ids[r, j] = -1
            seen.add(i)
    ids[0, [40, 95]], ids[0, 64], ids[1, [1, 33, 99]] = V - 1, V // 2, -1
    once = ids.clone()
    once[0, [40, 95, 64]] = -1
    loss, stats, grad, grad2 = check(R, x, once, values, 1.0, tail)
    twice = R.distill_fwd(x, ids, values, tail=tail)
    assert torch.equal(twice[0], loss) and torch.equal(twice[1], stats)
    assert torch.equal(R.distill_bwd(x, ids, values, None, stats, tail=tail), grad)
    assert torch.equal(R.distill_step(x, ids, values, tail=tail)[1], grad2)
    # copies whose rows lie as x's do: where a row begins in its first 16 bytes
    # decides in which order it is summed
    a, b = (torch.empty(2, V + 3, dtype=dtype, device="cuda")[:, 3:].copy_(x) for _ in range(2))
    assert torch.equal(R.distill_bwd(a, ids, values, None, stats, tail=tail, dstudent=a), grad)
    R.distill_step(b, ids, values, tail=tail, dstudent=b)
    assert torch.equal(b, grad2)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_tokens_and_short_lists(R, dtype, tail):
    """-inf and lowest-value logits, absent entries, an empty list, repeated
    ids (the first counts), rows of weight 0 whatever they hold."""
    g = gen(4)
    x = (2.0 * randn(g, 9, 3001)).to(dtype)
    ids, values = teacher_of(g, x, 12, 1.0, tail)
    drop = torch.rand(9, 3001, generator=g, device="cuda") < 0.4
    drop.scatter_(1, ids, False)
    x[0][drop[0]] = -INF
    x[1][drop[1]] = torch.finfo(dtype).min
    ids[2, 5:] = -1
    ids[3, [0, 7]] = -7
    values[4, 3] = -INF
    weight = torch.rand(9, generator=g, device="cuda")
    check(R, x, ids, values, 1.0, tail, weight)
    twice_ids, twice_values = ids.clone(), values.clone()
    twice_ids[5, [4, 9, 11]] = ids[5, 2]
    once_ids = twice_ids.clone()
    once_ids[5, [4, 9, 11]] = -1
    for f in (lambda i: R.distill_fwd(x, i, twice_values, tail=tail),
              lambda i: R.distill_step(x, i, twice_values, weight, tail=tail)):
        assert all(torch.equal(a, b) for a, b in zip(f(twice_ids), f(once_ids)))
    # weight 0: zeros, even for a row of NaN
    weight[[1, 6]] = 0.0
    x[6] = float("nan")
    loss, stats = R.distill_fwd(x, ids, values, tail=tail)
    grad = R.distill_bwd(x, ids, values, weight, stats, tail=tail)
    loss2, grad2 = R.distill_step(x, ids, values, weight, tail=tail)
    for gr in (grad, grad2):
        assert float(gr[[1, 6]].float().abs().max()) == 0
        assert bool(torch.isfinite(gr.float()).all())
    assert math.isnan(loss[6]) and math.isnan(loss2[6])


def test_rows_without_a_teacher_or_a_student(R):
    g = gen(5)
    x = 2.0 * randn(g, 6, 500)
    ids, values = teacher_of(g, x, 4, 1.0, False)
    ids[0] = -1
    values[1] = -INF
    x[2] = -INF
    x[3, 40] = float("nan")
    x[4, 41] = INF
    loss, stats = R.distill_fwd(x, ids, values)
    loss2, grad = R.distill_step(x, ids, values)
    bwd = R.distill_bwd(x, ids, values, None, stats)
    for r in (0, 1):
        assert float(loss[r]) == 0 and float(grad[r].abs().max()) == 0
        assert float(bwd[r].abs().max()) == 0
    assert float(loss[2]) == INF and float(grad[2].abs().max()) == 0
    assert float(bwd[2].abs().max()) == 0
    for r in (3, 4):
        assert math.isnan(loss[r]) and bool(torch.isnan(grad[r]).all())
        assert bool(torch.isnan(bwd[r]).all())
    assert bool(torch.isfinite(grad[5]).all()) and math.isfinite(loss[5])
    assert torch.equal(loss.isnan(), loss2.isnan())
    # the rest bucket with an empty list: teacher and student agree
    loss, _ = R.distill_fwd(x[5:], torch.full((1, 4), -1, device="cuda"), values[5:], tail=True)
    _, grad = R.distill_step(x[5:], torch.full((1, 4), -1, device="cuda"), values[5:], tail=True)
    assert float(loss.abs().max()) <= 1e-12 and float(grad.abs().max()) <= 1e-6


def test_id_past_the_vocabulary(R):
    g = gen(6)
    x = randn(g, 3, 64)
    ids, values = teacher_of(g, x, 4, 1.0, False)
    ids[1, 2] = 64
    loss, stats = R.distill_fwd(x, ids, values)
    assert math.isnan(loss[1]) and math.isfinite(loss[0]) and math.isfinite(loss[2])
    for grad in (R.distill_bwd(x, ids, values, None, stats), R.distill_step(x, ids, values)[1]):
        assert bool(torch.isnan(grad[1]).all()) and bool(torch.isfinite(grad[[0, 2]]).all())


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_small_losses_keep_their_digits(R, T):
    """A teacher that is the student moved by 1e-3: the loss is T^2 times about
    d^2 / 2 = 5e-7, with the relative error 2 e / |d| of the squared difference
    (e = 2e-6: logits of size 8), 1e-2 in all; the direct sum of p ln(p / q)
    would lose it.  A teacher equal to the student: (e^2 and the fp32 rounding
    of p_rest, 6e-8 squared) below 1e-10."""
    g = gen(7)
    x = 2.0 * randn(g, 4, 3000)
    for move, in ((1e-3,), (0.0,)):
        t = x + move * randn(g, 4, 3000)
        vals, ids = t.topk(100, dim=-1)
        vals = vals.double() / T - torch.logsumexp(t.double() / T, -1, keepdim=True)
        vals = vals.float()
        ref = reference(x, ids, vals, T, True)[0]
        loss, _ = R.distill_fwd(x, ids, vals, temperature=T, tail=True)
        if move:
            assert bool(((loss.double() - ref).abs() <= 1e-2 * ref).all())
        else:
            assert float(loss.abs().max()) <= 1e-10 * T * T
        assert bool((loss >= 0).all())


@pytest.mark.parametrize("tail", [False, True])
def test_peaked_student(R, tail):
    """One token with all but e^-100 of the student's probability, listed or
    not: ln q_rest comes from the rest's own maximum."""
    g = gen(8)
    x = randn(g, 2, 700)
    x[0, 5] = 110.0
    x[1, 6] = 110.0
    ids = torch.tensor([[5, 9, 11], [5, 9, 11]], device="cuda")
    values = torch.log(torch.tensor([[0.5, 0.2, 0.1], [0.3, 0.3, 0.3]], device="cuda"))
    loss, _, grad, _ = check(R, x, ids, values, 1.0, tail, None, 110.0)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(grad).all())


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(R, tail):
    """Five-point differences of the forward loss along random directions
    (step 0.05; truncation below h^4 = 6e-6 of the fifth derivative, rounding of
    the loss 1e-6 / h = 2e-5) within 2e-3 of the gradient's size."""
    g = gen(9)
    x = 2.0 * randn(g, 3, 1001)
    ids, values = teacher_of(g, x, 20, 1.5, tail)
    _, grad = R.distill_step(x, ids, values, temperature=1.5, tail=tail)
    h = 0.05
    for _ in range(3):
        v = randn(g, 3, 1001)
        f = [R.distill_fwd(x + k * h * v, ids, values, temperature=1.5, tail=tail)[0].double()
             for k in (-2, -1, 1, 2)]
        fd = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h)
        want = (grad.double() * v.double()).sum(-1)
        assert bool(((fd - want).abs() <= 2e-3 * grad.double().norm(dim=-1) + 1e-3).all())


def test_teacher_list_from_token_logprobs(R):
    """The list that token_logprobs gives for the teacher's logits, masked
    tokens' -1 entries among it, is what the loss takes."""
    g = gen(10)
    student, t = (2.0 * randn(g, 4, 2000)).bfloat16(), (2.0 * randn(g, 4, 2000)).bfloat16()
    t[1, 7:] = -INF  # seven allowed tokens: a list shorter than asked for
    _, _, lp, ids = R.token_logprobs(t, top=32, temperature=2.0)
    assert int((ids[1] < 0).sum()) == 25
    check(R, student, ids, lp, 2.0, True)


def test_no_rows(R):
    x = torch.empty(0, 50, device="cuda")
    ids, values = torch.empty(0, 3, dtype=torch.int64, device="cuda"), torch.empty(0, 3, device="cuda")
    loss, stats = R.distill_fwd(x, ids, values)
    assert loss.shape == (0,) and stats.shape == (0, 2)
    assert R.distill_step(x, ids, values)[1].shape == (0, 50)


def test_other_stream_and_graph(R):
    g = gen(11)
    x = (2.0 * randn(g, 16, 9001)).bfloat16()
    ids, values = teacher_of(g, x, 20, 1.0, True)
    want = R.distill_step(x, ids, values, tail=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = R.distill_step(x, ids, values, tail=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, stats = R.distill_fwd(x, ids, values, tail=True)
        grad = R.distill_bwd(x, ids, values, None, stats, tail=True)
        again = R.distill_step(x, ids, values, tail=True)
    first = None
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want)) and torch.equal(loss, want[0])
        assert first is None or torch.equal(first, grad)
        first = grad.clone()
