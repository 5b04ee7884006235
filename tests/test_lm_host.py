"""Host-side checks of the LayerNorm, logits and distillation entry points:
refusals before anything is launched; no GPU needed."""
import ctypes

import pytest
import torch

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
A, B, C = (ctypes.c_void_p(k << 32) for k in (1, 2, 3))  # addresses far apart


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention
    return retention


def ln_desc(R, n0=1, n1=4, d=64, dtype=1, eps=1e-5, sx=(0, 64), sg=(0, 64), so=(0, 64)):
    return R.LayerNormDesc(n0, n1, d, dtype, eps, sx, sg, so)


def lg_desc(R, n0=1, n1=4, V=100, dtype=1, T=1.0, top=3, id_bytes=8, tail=0, sx=(0, 100),
            sd=(0, 100)):
    return R.LogitsDesc(n0, n1, V, dtype, T, top, id_bytes, tail, sx, sd)


def test_layouts(R):
    assert ctypes.sizeof(R.LayerNormDesc) == 80 and R.LayerNormDesc.sx.offset == 32
    assert ctypes.sizeof(R.LogitsDesc) == 80 and R.LogitsDesc.sx.offset == 48
    assert R.MAX_TOP == 128


@pytest.mark.parametrize("bad", [
    dict(n0=-1), dict(n1=-2), dict(d=0), dict(d=(1 << 24) + 1), dict(dtype=2), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(sx=(0, -1)), dict(so=(0, 63)),
    dict(n0=1 << 30, n1=1 << 30), dict(n0=2, so=(255, 64)), dict(so=(0, 0))])
def test_layernorm_descriptors(R, bad):
    d = ctypes.byref(ln_desc(R, **bad))
    assert R.lib.retnet_layernorm_fwd(d, A, None, None, B, None, None, None) == EINVAL
    assert R.lib.retnet_layernorm_bwd(d, A, B, None, A, A, C, None, None, A, 1 << 40, None) == EINVAL


def test_layernorm_pointers_and_workspace(R):
    d = ctypes.byref(ln_desc(R))
    fwd = lambda x, y: R.lib.retnet_layernorm_fwd(d, x, None, None, y, None, None, None)
    assert fwd(None, B) == EINVAL and fwd(A, None) == EINVAL
    assert fwd(ctypes.c_void_p(A.value + 1), B) == EINVAL  # not on a bf16 value
    # y over a part of x, but not x itself
    assert fwd(A, ctypes.c_void_p(A.value + 128)) == EINVAL
    need = R.lib.retnet_layernorm_bwd_workspace_size(d)
    assert need >= 4 * 64 * 2 * 4
    bwd = lambda ws, n, dx=C, mean=A, rstd=A: R.lib.retnet_layernorm_bwd(
        d, A, B, None, mean, rstd, dx, None, None, ws, n, None)
    assert bwd(None, need) == EWORKSPACE and bwd(A, need - 1) == EWORKSPACE
    assert bwd(ctypes.c_void_p(A.value + 8), need) == EWORKSPACE
    assert bwd(A, need, mean=None) == EINVAL and bwd(A, need, rstd=None) == EINVAL
    assert bwd(A, need, dx=None) == EINVAL
    assert bwd(A, need, dx=ctypes.c_void_p(B.value + 64)) == EINVAL
    empty = ctypes.byref(ln_desc(R, n1=0))
    assert R.lib.retnet_layernorm_fwd(empty, None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("bad", [
    dict(n0=-1), dict(V=0), dict(V=(1 << 30) + 1), dict(dtype=7), dict(T=0.0), dict(T=-1.0),
    dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-20), dict(top=-1), dict(top=129),
    dict(id_bytes=2), dict(tail=2), dict(sx=(-1, 100)), dict(sd=(0, -5))])
def test_logits_descriptors(R, bad):
    d = ctypes.byref(lg_desc(R, **bad))
    assert R.lib.retnet_token_logprobs(d, A, B, C, None, None, None, None) == EINVAL
    assert R.lib.retnet_distill_fwd(d, A, B, C, C, C, None) == EINVAL
    assert R.lib.retnet_distill_bwd(d, A, B, C, None, C, C, None) == EINVAL
    assert R.lib.retnet_distill_step(d, A, B, C, None, C, None, C, None) == EINVAL


def test_logits_pointers(R):
    d = ctypes.byref(lg_desc(R))
    off = lambda p, n: ctypes.c_void_p(p.value + n)
    lp = lambda x, t, o: R.lib.retnet_token_logprobs(d, x, t, o, None, None, None, None)
    assert lp(None, B, C) == EINVAL
    assert lp(A, None, C) == EINVAL      # a log probability of no token
    assert lp(off(A, 1), B, C) == EINVAL and lp(A, off(B, 4), C) == EINVAL
    step = lambda x, ids, v, dx: R.lib.retnet_distill_step(d, x, ids, v, None, C, None, dx, None)
    assert step(None, B, C, C) == EINVAL and step(A, None, C, C) == EINVAL
    assert step(A, B, None, C) == EINVAL and step(A, B, C, None) == EINVAL
    assert step(A, B, C, off(A, 200)) == EINVAL          # over a part of x
    assert R.lib.retnet_distill_bwd(d, A, B, C, None, None, C, None) == EINVAL  # no statistics
    none = ctypes.byref(lg_desc(R, top=0))
    assert R.lib.retnet_distill_fwd(none, A, B, C, C, C, None) == EINVAL
    rows = ctypes.byref(lg_desc(R, sd=(0, 99)))          # gradient rows over one another
    assert R.lib.retnet_distill_step(rows, A, B, C, None, C, None, C, None) == EINVAL
    wide = ctypes.byref(lg_desc(R, V=(1 << 20) + 1, sx=(0, 1 << 21), sd=(0, 1 << 21)))
    assert R.lib.retnet_distill_fwd(wide, A, B, C, C, C, None) == EUNSUPPORTED


def test_binding_refusals(R):
    x = torch.zeros(3, 8)
    f32, ids = torch.zeros(3), torch.zeros(3, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        R.layernorm_fwd(x, out=x, mean=f32, rstd=f32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        R.token_logprobs(x, top=0, entropy=f32)
    with pytest.raises(ValueError, match="shape"):
        R.layernorm_fwd(x, torch.zeros(7))
    with pytest.raises(ValueError, match="contiguous fp32"):
        R.layernorm_fwd(x, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="dtype"):
        R.layernorm_fwd(x.half())
    with pytest.raises(ValueError, match="last dimension"):
        R.layernorm_fwd(torch.zeros(8, 3).t())
    with pytest.raises(ValueError, match="dy must have"):
        R.layernorm_bwd(x, x.bfloat16(), None, f32, f32)
    with pytest.raises(ValueError, match="do not fold"):
        R.layernorm_fwd(torch.zeros(3, 4, 5, 8).permute(2, 1, 0, 3),
                        out=torch.zeros(5, 4, 3, 8))
    with pytest.raises(TypeError, match="int32 or int64"):
        R.token_logprobs(x, f32)
    with pytest.raises(ValueError, match="tokens must be"):
        R.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="logprob needs tokens"):
        R.token_logprobs(x, logprob=f32)
    with pytest.raises(ValueError, match="ids must be"):
        R.distill_fwd(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(3, 2))
    with pytest.raises(ValueError, match="values must be"):
        R.distill_fwd(x, ids, torch.zeros(3, 3))
    with pytest.raises(ValueError, match="weight must be"):
        R.distill_bwd(x, ids, torch.zeros(3, 2), torch.zeros(3, dtype=torch.float64),
                      torch.zeros(3, 2), dstudent=x)
