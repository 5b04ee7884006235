"""Host-side checks of which tensors of the selective scan, causal convolution and
RMS norm calls may share memory; no GPU needed.  A call that passes its checks ends
at the launch (RET_ECUDA), since the tests' bodies run in processes of their own that
see no device: the addresses are none of a device's, and the library's last error
stays there.
"""
import os
import random
import subprocess
import sys

from tests.test_ssm_host import EINVAL, P, conv_bwd, conv_desc, off, rms_bwd, rms_desc, rms_quant, scan_bwd, scan_desc, scan_fwd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def alone(body):
    def run():
        import __graft_entry__
        __graft_entry__.build()
        code = ("from linear_recurrent_sequence_gb300 import retention as R\n"
                f"from tests import test_ssm_overlap_host as t\nt.{body.__name__}.body(R)")
        r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                           capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]

    run.__name__, run.__doc__, run.body = body.__name__, body.__doc__, body
    return run


@alone
def test_rmsnorm_gain_gradient_is_clear_of_the_rows(R):
    d = rms_desc(R)
    rows = 4 * 64 * 2  # bytes of [4, 64] bf16
    for k in range(3):  # h, dy, dh
        for at in (P[k], off(P[k], rows - 4), off(P[k], -252)):
            assert rms_bwd(R, d, dw=at) == EINVAL
        assert rms_bwd(R, d, dw=off(P[k], rows)) != EINVAL
    assert rms_bwd(R, d, dw=P[4]) == EINVAL and rms_bwd(R, d, dw=P[5]) == EINVAL


@alone
def test_conv_gradients_are_clear_of_the_rows(R):
    d = conv_desc(R)
    for k in (0, 5):  # x, dy
        assert conv_bwd(R, d, dw=P[k]) == EINVAL and conv_bwd(R, d, db=P[k]) == EINVAL and conv_bwd(R, d, dsi=P[k]) == EINVAL


@alone
def test_rows_of_other_widths_between(R):
    """y (8 values) in a buffer of rows of 40 that holds B and C (4 values) too."""
    rows = dict(sy=(200, 40), sB=(200, 40, 4), sC=(200, 40, 4), sdx=(200, 40))
    d = scan_desc(R, **rows)
    at = lambda col: off(P[10], 4 * col)
    for y, B, C, ok in ((8, 16, 20, True), (24, 16, 20, True), (0, 36, 8, True), (32, 0, 28, True), (9, 16, 20, False),
                        (13, 16, 20, False), (8, 15, 20, False), (17, 16, 30, False), (20, 0, 23, False),
                        (33, 40, 20, False), (32, 40, 20, True), (0, 40, 37, False)):
        got = scan_fwd(R, d, y=at(y), B=at(B), C=at(C))
        assert (got != EINVAL) == ok, (y, B, C)
        assert (scan_bwd(R, d, dy=P[22], dx=at(y), B=at(B), C=at(C)) != EINVAL) == ok, (y, B, C)
    # two groups reach from the first one's first state to the second one's last
    d = scan_desc(R, G=2, **dict(rows, sB=(200, 40, 14), sC=(200, 40, 14)))
    assert scan_fwd(R, d, y=at(18), B=at(0), C=P[4]) != EINVAL and scan_fwd(R, d, y=at(4), B=at(0), C=P[4]) == EINVAL
    # other strides
    assert scan_fwd(R, scan_desc(R, **dict(rows, sB=(400, 80, 4))), y=at(8), B=at(16)) == EINVAL


@alone
def test_rows_of_other_types_between(R):
    """e4m3 values in the second half of rows of 256 bytes that hold bf16 in the first."""
    d = rms_desc(R, sx=(0, 128), so=(0, 256))
    assert rms_quant(R, d, q=off(P[0], 128)) != EINVAL and rms_quant(R, d, q=off(P[0], 192)) != EINVAL
    for byte in (0, 127, 193):
        assert rms_quant(R, d, q=off(P[0], byte)) == EINVAL
    assert rms_quant(R, rms_desc(R, sx=(0, 128), so=(0, 128)), q=off(P[0], 128)) == EINVAL


@alone
def test_no_shared_value_passes(R):
    """Random rows of y and B: none passes that share a value, and all do that share
    none and whose strides keep rows of either width apart."""
    rng, passed, refused = random.Random(5), 0, 0
    for _ in range(4000):
        B, N, E, S = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 9), rng.randint(1, 9)
        s1 = rng.randint(E, 3 * E + S)
        s0 = (N - 1) * s1 + rng.randint(E, 3 * E + S)
        if rng.random() < 0.3:  # the batch inside the tokens
            s0 = rng.randint(E, E + S + 6)
            s1 = (B - 1) * s0 + rng.randint(E, 3 * E + S)
        shift = rng.randint(-(B * s0 + N * s1), B * s0 + N * s1)
        d = scan_desc(R, B=B, N=N, E=E, S=S, sy=(s0, s1), sB=(s0, s1, S))
        rows = [i * s0 + t * s1 for i in range(B) for t in range(N)]
        y = {r + c for r in rows for c in range(E)}
        shared = any(r + shift + c in y for r in rows for c in range(S))
        got = scan_fwd(R, d, y=P[10], B=off(P[10], 4 * shift)) != EINVAL
        assert not (got and shared), (B, N, E, S, s0, s1, shift)
        wide = max(E, S)
        apart = len({r + c for r in rows for c in range(wide)}) == len(rows) * wide
        inner, outer = (s1, s0) if s0 >= s1 else (s0, s1)
        nested = (N if s0 >= s1 else B) == 1 or (B if s0 >= s1 else N) == 1 or \
            outer >= ((N if s0 >= s1 else B) - 1) * inner + wide
        if not shared and apart and nested:
            assert got, (B, N, E, S, s0, s1, shift)
        passed, refused = passed + got, refused + (not got)
    assert passed > 500 and refused > 500
