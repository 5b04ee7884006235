"""GPU tests of operands that share one buffer without sharing a value: rows of
the output between, before or after rows of an input.  Results have to equal
those of separate tensors with the same strides, and what is between the rows
has to stay as it was; operands that do share values are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


# (shape of the buffer, the input's and the output's part of it)
LAYOUTS = {
    "beside": ((6, 2, 64), lambda b: b[:, 0], lambda b: b[:, 1]),
    "before": ((6, 2, 64), lambda b: b[:, 1], lambda b: b[:, 0]),
    "halves of columns": ((5, 7, 130), lambda b: b[..., :65], lambda b: b[..., 65:]),
    "halves of a sequence": ((3, 10, 72), lambda b: b[:, :5], lambda b: b[:, 5:]),
    "second half first": ((3, 10, 72), lambda b: b[:, 5:], lambda b: b[:, :5]),
    "batch inside": ((4, 6, 48), lambda b: b.transpose(0, 1)[:, :2], lambda b: b.transpose(0, 1)[:, 2:]),
    "every other row": ((12, 40), lambda b: b[::2], lambda b: b[1::2]),
}


def buffers(layout, dtype):
    shape, a, b = LAYOUTS[layout]
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    buf = torch.randn(*shape, generator=g, device="cuda").to(dtype)
    return buf, a, b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_layernorm_beside_its_input(R, layout, dtype):
    buf, a, b = buffers(layout, dtype)
    far = buf.clone()
    x, y = a(buf), b(buf)
    kept = x.clone()
    want, mean, rstd = R.layernorm_fwd(a(far), out=b(torch.empty_like(far)))
    got = R.layernorm_fwd(x, out=y)
    assert torch.equal(y, want) and torch.equal(x, kept)
    assert torch.equal(got[1], mean) and torch.equal(got[2], rstd)
    buf.copy_(far)
    dx = R.layernorm_bwd(a(far), a(far), None, mean, rstd, dx=b(torch.empty_like(far)))[0]
    R.layernorm_bwd(x, x, None, mean, rstd, dx=y)
    assert torch.equal(y, dx) and torch.equal(x, kept)


@pytest.mark.parametrize("layout", list(LAYOUTS))
def test_distillation_gradient_beside_the_logits(R, layout):
    buf, a, b = buffers(layout, torch.float32)
    x, y = a(buf), b(buf)
    lead = x.shape[:-1]
    ids = torch.zeros(*lead, 2, dtype=torch.int64, device="cuda")
    ids[..., 1] = 9
    values = torch.zeros(*lead, 2, device="cuda")
    far = buf.clone()
    kept = x.clone()
    loss, want = R.distill_step(a(far), ids, values, dstudent=b(torch.empty_like(far)))
    got, _ = R.distill_step(x, ids, values, dstudent=y)
    assert torch.equal(y, want) and torch.equal(x, kept) and torch.equal(got, loss)


def test_shared_values_are_refused(R):
    buf = torch.randn(6, 200, device="cuda")
    kept = buf.clone()
    for x, y in ((buf[:, :100], buf[:, 99:199]), (buf[:, 50:150], buf[:, :100]), (buf[:5, :100], buf[1:, :100]),
                 (buf[:3, :100], buf[1:6:2, :100]), (buf[:, :100], buf[:, 8:108])):
        with pytest.raises(R.RetentionError, match="EINVAL"):
            R.layernorm_fwd(x, out=y)
        ids, values = torch.zeros(x.shape[0], 1, dtype=torch.int64, device="cuda"), torch.zeros(x.shape[0], 1, device="cuda")
        with pytest.raises(R.RetentionError, match="EINVAL"):
            R.distill_step(x, ids, values, dstudent=y)
    cube = torch.randn(4, 6, 30, device="cuda")
    for x, y in ((cube[:, :4], cube[:, 2:]), (cube[:3, :4], cube[1:, 2:]), (cube[:3, 2:], cube[1:, :4]),
                 (cube[:2, :, 10:], cube[1:3, :, :20])):
        with pytest.raises(R.RetentionError, match="EINVAL"):
            R.layernorm_fwd(x, out=y)
    assert torch.equal(buf, kept)
