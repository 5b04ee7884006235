"""Host-side checks of which tensors of the selective scan, causal convolution and
RMS norm calls may share memory; no GPU needed: a call that passes its checks ends
at the launch, which there is no device for (RET_ECUDA), a refused one before it.
"""
import ctypes

import pytest
import torch

from tests.test_ssm_host import EINVAL, P, R, conv_bwd, conv_desc, off, rms_bwd, rms_desc  # noqa: F401 (R: fixture)


@pytest.fixture(autouse=True)
def no_device():
    if torch.cuda.is_available():
        pytest.skip("the addresses are no device's")


def test_rmsnorm_gain_gradient_is_clear_of_the_rows(R):
    d = rms_desc(R)
    rows = 4 * 64 * 2  # bytes of [4, 64] bf16
    for k in range(3):  # h, dy, dh
        for at in (P[k], off(P[k], rows - 4), off(P[k], -252)):
            assert rms_bwd(R, d, dw=at) == EINVAL
        assert rms_bwd(R, d, dw=off(P[k], rows)) != EINVAL
    assert rms_bwd(R, d, dw=P[4]) == EINVAL and rms_bwd(R, d, dw=P[5]) == EINVAL


def test_conv_gradients_are_clear_of_the_rows(R):
    d = conv_desc(R)
    for k in (0, 5):  # x, dy
        assert conv_bwd(R, d, dw=P[k]) == EINVAL and conv_bwd(R, d, db=P[k]) == EINVAL and conv_bwd(R, d, dsi=P[k]) == EINVAL
