"""Host-side checks of the selective scan, causal convolution and RMS norm entry
points: refusals before anything is launched, and the norm's border cases; no
GPU needed."""
import ctypes

import pytest
import torch

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
P = [ctypes.c_void_p((k + 1) << 36) for k in range(24)]  # addresses far apart


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention
    return retention


def off(p, n):
    return ctypes.c_void_p(p.value + n)


def scan_desc(R, B=2, N=5, E=8, S=4, G=1, dtype=0, softplus=1, len_bytes=4, **strides):
    rows = (40, 8)
    d = {k: rows for k in ("sx", "sdt", "sz", "sy", "sdy", "sdx", "sddt", "sdz")}
    d.update(sB=(20, 4, 4), sC=(20, 4, 4))
    d.update(strides)
    return R.ScanDesc(B, N, E, S, G, dtype, softplus, len_bytes, *(d[k] for k in (
        "sx", "sdt", "sz", "sy", "sdy", "sdx", "sddt", "sdz", "sB", "sC")))


def test_layouts(R):
    assert ctypes.sizeof(R.ScanDesc) == 208 and R.ScanDesc.sx.offset == 32 and R.ScanDesc.sB.offset == 160
    assert ctypes.sizeof(R.ConvDesc) == 80 and R.ConvDesc.sx.offset == 32
    assert ctypes.sizeof(R.RmsNormDesc) == 112 and R.RmsNormDesc.sx.offset == 32
    assert R.MAX_STATES == 64


def scan_fwd(R, d, x=P[0], dt=P[1], A=P[2], B=P[3], C=P[4], D=P[5], z=P[6], bias=P[7], h_in=P[8], lengths=P[9],
             y=P[10], h_out=P[11], ws=None, n=0):
    return R.lib.retnet_selective_scan_fwd(ctypes.byref(d), x, dt, A, B, C, D, z, bias, h_in, lengths, y, h_out, ws, n, None)


def scan_step(R, d, x=P[0], dt=P[1], A=P[2], B=P[3], C=P[4], D=P[5], z=P[6], bias=P[7], h_in=P[8], y=P[10], h_out=P[11]):
    return R.lib.retnet_selective_scan_step(ctypes.byref(d), x, dt, A, B, C, D, z, bias, h_in, y, h_out, None)


def scan_bwd(R, d, x=P[0], dt=P[1], A=P[2], B=P[3], C=P[4], D=P[5], z=P[6], bias=P[7], h_in=P[8], lengths=P[9], dy=P[10],
             dh=P[11], dx=P[12], ddt=P[13], dA=P[14], dB=P[15], dC=P[16], dD=P[17], dz=P[18], dbias=P[19], dh_in=P[20],
             ws=P[21], n=1 << 40):
    return R.lib.retnet_selective_scan_bwd(ctypes.byref(d), x, dt, A, B, C, D, z, bias, h_in, lengths, dy, dh, dx, ddt, dA,
                                           dB, dC, dD, dz, dbias, dh_in, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=65536), dict(N=-1), dict(N=(1 << 24) + 1), dict(E=0), dict(E=(1 << 24) + 1), dict(S=0), dict(S=65),
    dict(G=0), dict(G=3), dict(dtype=2), dict(softplus=2), dict(len_bytes=2), dict(sx=(40, -8)), dict(sB=(-1, 4, 4)),
    dict(sC=(20, 4, -4)), dict(sdt=(1 << 46, 8))])
def test_scan_descriptors(R, bad):
    d = scan_desc(R, **bad)
    assert scan_fwd(R, d) == EINVAL and scan_bwd(R, d) == EINVAL
    assert scan_step(R, scan_desc(R, **dict(dict(N=1), **bad))) == EINVAL


def test_scan_pointers_and_workspace(R):
    d = scan_desc(R)
    for name in ("x", "dt", "A", "B", "C", "y"):
        assert scan_fwd(R, d, **{name: None}) == EINVAL
        assert scan_fwd(R, d, **{name: off(P[12], 2)}) == EINVAL  # not on an fp32 value
    for name in ("x", "dt", "A", "B", "C", "dy", "dx", "ddt", "dB", "dC", "dz"):
        assert scan_bwd(R, d, **{name: None}) == EINVAL
    for name in ("h_in", "bias", "D", "lengths", "dh", "dA", "dD", "dbias", "dh_in"):
        assert scan_bwd(R, d, **{name: off(P[22], 2)}) == EINVAL
    need = R.lib.retnet_selective_scan_bwd_workspace_size(ctypes.byref(d))
    assert need >= 2 * 2 * 8 * 4 * 4
    assert scan_bwd(R, d, ws=None, n=0) == EWORKSPACE and scan_bwd(R, d, n=need - 1) == EWORKSPACE
    assert scan_bwd(R, d, ws=off(P[21], 8)) == EWORKSPACE
    assert scan_fwd(R, scan_desc(R, B=0)) == 0
    step = scan_desc(R, N=1)
    for name in ("x", "dt", "A", "B", "C", "y", "h_in", "h_out"):
        assert scan_step(R, step, **{name: None}) == EINVAL
    assert scan_step(R, scan_desc(R, N=2)) == EINVAL


def test_scan_overlaps(R):
    d = scan_desc(R)
    rows = 2 * 40 * 4  # bytes of [2, 5, 8] fp32
    assert scan_fwd(R, d, y=P[0]) == EINVAL and scan_fwd(R, d, y=off(P[0], rows - 4)) == EINVAL
    assert scan_fwd(R, d, y=P[6]) == EINVAL and scan_fwd(R, d, y=P[2]) == EINVAL
    assert scan_fwd(R, d, h_out=P[8]) == EINVAL          # in place only for one token
    assert scan_fwd(R, d, h_out=P[10]) == EINVAL         # over y
    assert scan_step(R, scan_desc(R, N=1), h_out=off(P[8], 4)) == EINVAL
    assert scan_bwd(R, d, dx=P[0]) == EINVAL and scan_bwd(R, d, dx=P[13]) == EINVAL
    assert scan_bwd(R, d, dA=P[2]) == EINVAL and scan_bwd(R, d, dB=P[16]) == EINVAL
    assert scan_bwd(R, d, dh_in=P[11]) == EINVAL
    # rows over one another
    assert scan_fwd(R, scan_desc(R, sy=(40, 7))) == EINVAL and scan_bwd(R, scan_desc(R, sdz=(8, 8))) == EINVAL


def conv_desc(R, B=2, N=5, E=8, W=4, dtype=0, silu=1, len_bytes=4, sx=(40, 8), sg=(40, 8), so=(40, 8)):
    return R.ConvDesc(B, N, E, W, dtype, silu, len_bytes, sx, sg, so)


def conv_fwd(R, d, x=P[0], w=P[1], b=P[2], state_in=P[3], lengths=P[4], y=P[5], state_out=P[6]):
    return R.lib.retnet_causal_conv_fwd(ctypes.byref(d), x, w, b, state_in, lengths, y, state_out, None)


def conv_bwd(R, d, x=P[0], w=P[1], b=P[2], state_in=P[3], lengths=P[4], dy=P[5], dso=P[6], dx=P[7], dw=P[8], db=P[9],
             dsi=P[10], ws=P[11], n=1 << 40):
    return R.lib.retnet_causal_conv_bwd(ctypes.byref(d), x, w, b, state_in, lengths, dy, dso, dx, dw, db, dsi, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(B=70000), dict(N=-1), dict(E=0), dict(W=1), dict(W=5), dict(dtype=3), dict(silu=2), dict(len_bytes=1),
    dict(sx=(-1, 8)), dict(sg=(0, -8)), dict(so=(40, 7)), dict(so=(0, 8))])
def test_conv_descriptors(R, bad):
    d = conv_desc(R, **bad)
    assert conv_fwd(R, d) == EINVAL and conv_bwd(R, d) == EINVAL


def test_conv_pointers_overlaps_and_workspace(R):
    d = conv_desc(R)
    for name in ("x", "w", "y"):
        assert conv_fwd(R, d, **{name: None}) == EINVAL
    for name in ("x", "w", "b", "state_in", "lengths", "y", "state_out"):
        assert conv_fwd(R, d, **{name: off(P[12], 2)}) == EINVAL
    for name in ("x", "w", "dy", "dx"):
        assert conv_bwd(R, d, **{name: None}) == EINVAL
    assert conv_fwd(R, d, y=P[0]) == EINVAL and conv_fwd(R, d, state_out=off(P[3], 4)) == EINVAL
    assert conv_fwd(R, d, state_out=P[5]) == EINVAL
    assert conv_bwd(R, d, dx=P[5]) == EINVAL and conv_bwd(R, d, dsi=P[6]) == EINVAL and conv_bwd(R, d, dw=P[9]) == EINVAL
    need = R.lib.retnet_causal_conv_bwd_workspace_size(ctypes.byref(d))
    assert need >= 2 * 8 * 5 * 4 and conv_bwd(R, d, n=need - 1) == EWORKSPACE and conv_bwd(R, d, ws=None) == EWORKSPACE
    assert conv_fwd(R, conv_desc(R, B=0)) == 0


def rms_desc(R, n0=1, n1=4, d=64, dtype=1, eps=1e-5, group=0, sx=(0, 64), sr=(0, 64), sh=(0, 64), sg=(0, 64), so=(0, 64)):
    return R.RmsNormDesc(n0, n1, d, dtype, eps, group, sx, sr, sh, sg, so)


def rms_fwd(R, d, x=P[0], r=P[1], w=P[2], h=P[3], y=P[4], rstd=P[5]):
    return R.lib.retnet_rmsnorm_fwd(ctypes.byref(d), x, r, w, h, y, rstd, None)


def rms_quant(R, d, x=P[0], r=P[1], w=P[2], h=P[3], q=P[4], scales=P[5]):
    return R.lib.retnet_rmsnorm_quant(ctypes.byref(d), x, r, w, h, q, scales, None)


def rms_bwd(R, d, h=P[0], dy=P[1], dh=P[2], w=P[3], rstd=P[4], dx=P[5], dw=P[6], ws=P[7], n=1 << 40):
    return R.lib.retnet_rmsnorm_bwd(ctypes.byref(d), h, dy, dh, w, rstd, dx, dw, ws, n, None)


@pytest.mark.parametrize("bad", [
    dict(n0=-1), dict(n1=-2), dict(d=0), dict(d=(1 << 24) + 1), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(group=-8), dict(group=12), dict(sx=(0, -1)), dict(so=(0, 63)), dict(n0=1 << 30, n1=1 << 30)])
def test_rmsnorm_descriptors(R, bad):
    d = rms_desc(R, **bad)
    assert rms_fwd(R, d) == EINVAL and rms_quant(R, d) == EINVAL and rms_bwd(R, d) == EINVAL


def test_rmsnorm_pointers_and_overlaps(R):
    d = rms_desc(R)
    for name in ("x", "h", "y"):
        assert rms_fwd(R, d, **{name: None}) == EINVAL
    assert rms_quant(R, d, scales=None) == EINVAL and rms_quant(R, d, q=None) == EINVAL
    assert rms_fwd(R, d, x=off(P[0], 1)) == EINVAL and rms_fwd(R, d, rstd=off(P[5], 2)) == EINVAL
    assert rms_fwd(R, d, h=off(P[0], 128)) == EINVAL and rms_fwd(R, d, y=P[3]) == EINVAL
    assert rms_fwd(R, rms_desc(R, sh=(0, 63))) == EINVAL
    assert rms_quant(R, d, q=P[0]) == EINVAL and rms_quant(R, d, scales=P[4]) == EINVAL
    for name in ("h", "dy", "rstd", "dx"):
        assert rms_bwd(R, d, **{name: None}) == EINVAL
    assert rms_bwd(R, d, dx=off(P[1], 64)) == EINVAL and rms_bwd(R, d, dw=P[3]) == EINVAL
    need = R.lib.retnet_rmsnorm_bwd_workspace_size(ctypes.byref(d))
    assert rms_bwd(R, d, n=need - 1) == EWORKSPACE and rms_bwd(R, d, ws=None) == EWORKSPACE
    assert rms_fwd(R, rms_desc(R, n1=0), None, None, None, None, None, None) == 0


def test_binding_refusals(R):
    x, A, bc = torch.zeros(2, 3, 8), torch.zeros(8, 4), torch.zeros(2, 3, 1, 4)
    fwd = lambda **k: R.selective_scan_fwd(*[k.pop(n, v) for n, v in (("x", x), ("dt", x), ("A", A), ("B", bc), ("C", bc))], **k)
    with pytest.raises(ValueError, match="CUDA tensor"):
        fwd()
    with pytest.raises(TypeError, match="dtype"):
        fwd(x=x.half(), dt=x.half())
    with pytest.raises(ValueError, match="dt must have"):
        fwd(dt=x.bfloat16())
    with pytest.raises(ValueError, match="contiguous fp32"):
        fwd(A=A.bfloat16())
    with pytest.raises(ValueError, match="contiguous fp32"):
        fwd(A=torch.zeros(4, 8).t())
    with pytest.raises(ValueError, match="B must have"):
        fwd(B=torch.zeros(2, 3, 1, 5))
    with pytest.raises(ValueError, match="equal groups"):
        fwd(B=torch.zeros(2, 3, 3, 4), C=torch.zeros(2, 3, 3, 4))
    with pytest.raises(ValueError, match="states must be contiguous"):
        fwd(C=torch.zeros(2, 3, 1, 8)[..., ::2])
    with pytest.raises(ValueError, match="channels must be contiguous"):
        fwd(z=torch.zeros(2, 8, 3).transpose(1, 2))
    with pytest.raises(TypeError, match="int32 or int64"):
        fwd(lengths=torch.zeros(2))
    with pytest.raises(ValueError, match="lengths must be"):
        fwd(lengths=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="h_in must be"):
        fwd(h_in=torch.zeros(2, 8, 5))
    with pytest.raises(ValueError, match="x must be"):
        R.selective_scan_step(x, x, A, bc, bc, torch.zeros(2, 8, 4))
    with pytest.raises(ValueError, match="dy must have"):
        R.selective_scan_bwd(x, x, A, bc, bc, torch.zeros(2, 3, 9))
    with pytest.raises(ValueError, match="dB must be"):
        R.selective_scan_bwd(x, x, A, bc, bc, x, dB=torch.zeros(2, 3, 1, 5))
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        R.causal_conv_fwd(x, w)
    with pytest.raises(ValueError, match="state_in must be"):
        R.causal_conv_fwd(x, w, state_in=torch.zeros(2, 4, 8))
    with pytest.raises(ValueError, match="w must be"):
        R.causal_conv_bwd(x, torch.zeros(7, 4), None, x)
    with pytest.raises(ValueError, match="residual_out needs"):
        R.rmsnorm_fwd(x, residual_out=x)
    with pytest.raises(ValueError, match="multiple of 8"):
        R.rmsnorm_quant(x, group=12)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        R.rmsnorm_quant(x, out=torch.zeros(2, 3, 8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dh must have"):
        R.rmsnorm_bwd(x, x, None, torch.zeros(2, 3), dh=x[:1])


def test_checks_are_found_by_shapes_and_not_by_tensors(R, monkeypatch):
    """Options and addresses are those of each call; a tensor of another layout
    is checked anew."""
    given = []

    class Library:
        def __init__(self, lib):
            self.lib = lib

        def __getattr__(self, name):
            if "workspace_size" in name or "status" in name:
                return getattr(self.lib, name)

            def call(desc, *args):
                d = desc._obj
                given.append((type(d).from_buffer_copy(ctypes.string_at(ctypes.addressof(d), ctypes.sizeof(d))), args))
                return 0
            return call

    monkeypatch.setattr(R, "lib", Library(R.lib))
    monkeypatch.setattr(R, "_ptrs", lambda *ts: [None if t is None else t.data_ptr() for t in ts])
    monkeypatch.setattr(R, "_stream", lambda s: None)
    A, bc = torch.zeros(8, 4), torch.zeros(2, 3, 1, 4)
    for soft in (True, False, torch.tensor(True)):
        x = torch.zeros(2, 3, 8)
        R.selective_scan_fwd(x, x, A, bc, bc, softplus=soft)
        assert given[-1][0].softplus == int(bool(soft)) and given[-1][1][0] == x.data_ptr()
    wide = torch.zeros(2, 3, 20)
    R.selective_scan_fwd(wide[..., 3:11], x, A, bc, bc)
    assert tuple(given[-1][0].sx) == (60, 20) and tuple(given[-1][0].sdt) == (24, 8)
    n = torch.tensor([1, 2])
    R.selective_scan_fwd(x, x, A, bc, bc, lengths=n)
    assert given[-1][0].len_bytes == 8
    R.selective_scan_fwd(x, x, A, bc, bc, lengths=n.int())
    assert given[-1][0].len_bytes == 4
    with pytest.raises(ValueError, match="channels must be contiguous"):
        R.selective_scan_fwd(torch.zeros(2, 8, 3).transpose(1, 2), x, A, bc, bc)
    w = torch.zeros(8, 3)
    R.causal_conv_fwd(x, w, silu=False)
    assert (given[-1][0].silu, given[-1][0].W) == (0, 3)
    eps = torch.tensor(0.5)
    for want in (0.5, 0.25):
        eps.fill_(want)
        R.rmsnorm_fwd(x, eps=eps)
        assert given[-1][0].eps == want
    R._scan_plan.cache_clear()
    R._conv_plan.cache_clear()
    R._rms_plan.cache_clear()
