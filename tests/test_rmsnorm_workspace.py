"""The workspace of the RMS norm's gradients: as many rows of sums as CTAs write,
and no byte behind it written."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention
    return retention


def size(R, rows, d, dtype):
    r = (0, d)
    desc = R.RmsNormDesc(1, rows, d, dtype, 0.0, 0, r, r, r, r, r)
    return int(R.lib.retnet_rmsnorm_bwd_workspace_size(ctypes.byref(desc)))


# (rows, d, bf16: CTAs an SM that are started for rows of this width; None: two
# passes, 64 rows of sums in all and a value a row)
SIZES = [(1 << 16, 8192, True, 2), (1 << 16, 8192, False, 2), (1 << 16, 4096, True, 4), (1 << 16, 4000, False, 4),
         (1 << 16, 1000, True, 16), (1 << 16, 64, False, 16), (2432, 1 << 20, True, None), (2432, 1 << 20, False, None),
         (5000, 8200, False, None), (1 << 16, 16384, True, 2), (30, 1 << 20, True, None), (3, 4096, True, 4)]


@pytest.mark.parametrize("rows,d,bf16,ctas", SIZES)
def test_size(R, rows, d, bf16, ctas):
    """(Without a device one SM is counted.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1
    groups = 64 if ctas is None else ctas * sms
    if bf16 and 8192 < d <= 16384:  # (rows off the 16-byte boundary take two passes)
        groups = max(groups, 64)
    need = size(R, rows, d, R.BF16 if bf16 else R.F32)
    assert need <= (min(rows, groups) * d + rows) * 4 + 512


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,shift", [(5000, 64, 0), (3000, 257, 1), (4000, 1000, 0), (1300, 4096, 0), (1300, 4096, 1),
                                          (700, 8192, 0), (700, 8200, 0), (400, 16384, 0), (400, 16384, 1), (130, 40000, 0)])
def test_no_byte_behind_it(R, dtype, rows, d, shift):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + d)
    wide = lambda: torch.randn(rows, d + shift, generator=g, device="cuda").to(dtype)[:, shift:]
    h, dy, w = wide(), wide(), torch.rand(d, generator=g, device="cuda")
    _, _, rstd = R.rmsnorm_fwd(h, w)
    want = R.rmsnorm_bwd(h, dy, w, rstd)
    need = size(R, rows, d, R.BF16 if dtype == torch.bfloat16 else R.F32)
    buf = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    got = R.rmsnorm_bwd(h, dy, w, rstd, workspace=buf[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((buf[need:] == 0xA5).all())
    with pytest.raises(R.RetentionError):
        R.rmsnorm_bwd(h, dy, w, rstd, workspace=buf[:need - 1])
