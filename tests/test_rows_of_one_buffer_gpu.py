"""Outputs of the selective scan and the RMS norm in the columns beside their
inputs of other widths and types, in one buffer: the results of separate tensors, and
nothing else of the buffer changes."""
import pytest
import torch

from tests.test_scan_gpu import BF16, F32, R, gen, problem, rand  # noqa: F401 (R: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("E,S,G,first", [(48, 16, 1, 0), (41, 7, 1, 3), (64, 8, 2, 8)])
def test_scan(R, dtype, E, S, G, first):
    B, N = 3, 90
    args, kw = problem(E, B, N, E, S, G, dtype)
    y, h = R.selective_scan_fwd(*args, **kw)
    dy = rand(gen(1), B, N, E, dtype=dtype)
    want = R.selective_scan_bwd(*args, dy, **kw)
    buf = torch.full((B, N, first + E + 2 * G * S + E + 3), 7.0, dtype=dtype, device="cuda")
    at = first + E
    Bm, Cm = (buf[..., c:c + G * S].unflatten(-1, (G, S)) for c in (at, at + G * S))
    Bm.copy_(args[3])
    Cm.copy_(args[4])
    left, right = buf[..., first:at], buf[..., at + 2 * G * S:at + 2 * G * S + E]
    one = [*args[:3], Bm, Cm]
    for out in (left, right):
        got, h2 = R.selective_scan_fwd(*one, **kw, out=out)
        assert got is out and torch.equal(out, y) and torch.equal(h2, h)
    grads = R.selective_scan_bwd(*one, dy, **kw, dx=left, ddt=right)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert torch.equal(Bm, args[3]) and torch.equal(Cm, args[4])
    assert bool((buf[..., :first] == 7).all()) and bool((buf[..., at + 2 * G * S + E:] == 7).all())


@pytest.mark.parametrize("rows,d", [(40, 256), (7, 97), (3, 20000)])
def test_e4m3_beside_bf16(R, rows, d):
    g = gen(rows)
    x = rand(g, rows, d, dtype=BF16)
    wide = (2 * d + d + 15) // 16 * 16
    buf = torch.full((rows, wide), 9, dtype=torch.uint8, device="cuda")
    xin = buf.view(BF16)[:, :d]
    xin.copy_(x)
    out = buf[:, 2 * d:3 * d].view(torch.float8_e4m3fn)
    q, s, _ = R.rmsnorm_quant(xin, group=32, out=out)
    want, ws, _ = R.rmsnorm_quant(x.clone(), group=32)
    same = d % 16 == 0  # (else rows of another alignment, whose sums have another order)
    assert torch.equal(xin, x) and bool((buf[:, 3 * d:] == 9).all())
    if same:
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)
    else:
        assert bool(((s - ws).abs() <= 2.0 ** -16 * ws).all())
