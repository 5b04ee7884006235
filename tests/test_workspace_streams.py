"""Workspaces that the binding makes for a call on a stream of the caller's.

They have to be allocated (and zeroed) in that stream's order: the caching
allocator gives a freed block to the next allocation of the stream it was
allocated on, which for any other stream may be while the call's kernels still
use it.  On the CPU the library is replaced by a recorder; on the GPU, long
work is queued on the side stream before the call and buffers of the
workspace's size are allocated and filled on the current stream after it.
"""
import contextlib
import ctypes
import types

import pytest
import torch


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention
    return retention


class Recorder:
    """Stands for torch's stream context, the allocations that make workspaces
    and the library: which stream was current at each allocation of bytes."""

    def __init__(self, R, monkeypatch):
        self.current, self.made, self.given = None, {}, []
        real_empty, real_zeros = torch.empty, torch.zeros

        def note(real):
            def make(*a, **k):
                t = real(*a, **k)
                if t.dtype is torch.uint8:
                    self.made[t.data_ptr()] = self.current
                return t
            return make

        @contextlib.contextmanager
        def stream_context(s):
            before, self.current = self.current, s
            try:
                yield
            finally:
                self.current = before

        class Library:
            def __init__(self, lib):
                self.lib = lib

            def __getattr__(self, name):
                if "workspace_size" in name or "status" in name:
                    return getattr(self.lib, name)

                def call(*args):
                    addresses = [getattr(a, "value", a) for a in args]
                    recorder.given.append([recorder.made[a] for a in addresses
                                           if isinstance(a, int) and a in recorder.made])
                    return 0
                return call

        recorder = self
        monkeypatch.setattr(torch, "empty", note(real_empty))
        monkeypatch.setattr(torch, "zeros", note(real_zeros))
        monkeypatch.setattr(torch.cuda, "stream", stream_context)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a, **k: FakeStream(handle))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(7))
        monkeypatch.setattr(R, "lib", Library(R.lib))
        monkeypatch.setattr(R, "_ptr", lambda t: None if t is None else ctypes.c_void_p(t.data_ptr()))
        monkeypatch.setattr(R, "_ptrs", lambda *ts: [None if t is None else t.data_ptr() for t in ts])


def FakeStream(handle):
    """A stream as the binding sees it, without a device."""
    return types.SimpleNamespace(cuda_stream=handle)


def calls(R, dev="cpu"):
    """name -> f(stream): one call of each entry point that makes a workspace."""
    f32 = lambda *s: torch.randn(*s, device=dev)
    b16 = lambda *s: (0.2 * torch.randn(*s, device=dev)).bfloat16()
    q, k, v = b16(1, 2, 64, 64), b16(1, 2, 64, 64), b16(1, 2, 64, 128)
    gam = [0.9, 0.95]
    x, w = f32(40, 64), f32(64)
    stat = f32(40)
    X = b16(1, 16, 128)
    W = dict(WQ=b16(128, 128), WK=b16(128, 128), WV=b16(128, 256), WG=b16(128, 256), WO=b16(256, 128))
    shape = dict(H=2, d_k=64, d_v=128, gamma=gam)
    ln, ffn = [f32(128), f32(128)], [b16(128, 256), b16(256, 128)]
    layer = dict(zip(R.LAYER_KEYS, [*ln, *W.values(), *ln, *ffn]))
    S, token = f32(1, 2, 64, 128), b16(1, 128)
    return {
        "layernorm_bwd": lambda s: R.layernorm_bwd(x, x, w, stat, stat, stream=s),
        "chunkwise_fwd": lambda s: R.chunkwise_fwd(q, k, v, gam, stream=s),
        "chunkwise_state": lambda s: R.chunkwise_state(k, v, gam, stream=s),
        "chunkwise_bwd": lambda s: R.chunkwise_bwd(q, k, v, v, gam, stream=s),
        "parallel_fwd": lambda s: R.parallel_fwd(q, k, v, gam, stream=s),
        "recurrent_step": lambda s: R.recurrent_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], S, gam, pos=0, stream=s),
        "msr_layer_fwd": lambda s: R.msr_layer_fwd(X, **W, **shape, stream=s),
        "retnet_block_fwd": lambda s: R.retnet_block_fwd(X, *ln, *W.values(), *ln, *ffn, **shape, stream=s),
        "retnet_decode_step": lambda s: R.retnet_decode_step(token, [layer], [S], **shape, pos=0, stream=s),
        "gemm_bf16": lambda s: R.gemm_bf16(W["WQ"], W["WV"], stream=s),
    }


NAMES = ["layernorm_bwd", "chunkwise_fwd", "chunkwise_state", "chunkwise_bwd", "parallel_fwd", "recurrent_step",
         "msr_layer_fwd", "retnet_block_fwd", "retnet_decode_step", "gemm_bf16"]


@pytest.mark.parametrize("name", NAMES)
def test_allocated_in_the_order_of_its_stream(R, name, monkeypatch):
    make = calls(R)[name]
    rec = Recorder(R, monkeypatch)
    side = FakeStream(9)
    make(side)
    assert rec.given and rec.given[-1], "the call was given no workspace of the binding's"
    # (the stream itself, or one made of its handle)
    assert all(s is not None and s.cuda_stream == 9 for s in rec.given[-1])
    assert rec.current is None


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_blocks_are_not_given_away_while_in_use(R, name):
    """Equal to the call by itself, and the buffers keep what was written to
    them, although the call's kernels run only long after it returned."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.manual_seed(3)
    make = calls(R, "cuda")[name]

    def flat(out):
        return [t.clone() for t in (out if isinstance(out, tuple) else (out,)) if t is not None]

    torch.cuda.synchronize()
    want = flat(make(None))
    torch.cuda.synchronize()
    moves_on = name in ("recurrent_step", "retnet_decode_step")  # the state: one turn from the same one
    if moves_on:
        torch.manual_seed(3)
        make = calls(R, "cuda")[name]
    busy = torch.randn(6144, 6144, device="cuda").bfloat16()
    sizes = [256 << j for j in range(16)]
    side = torch.cuda.Stream()
    for _ in range(2):  # (the first turn leaves freed blocks behind)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                busy @ busy
        got = make(side)
        filled = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        if moves_on:
            break
    assert all(torch.equal(a, b) for a, b in zip(flat(got), want))
    assert all(bool((t == 0xA5).all()) for t in filled)
