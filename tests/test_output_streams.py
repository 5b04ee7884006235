"""Outputs that the binding allocates for a call on a stream of the caller's.

They belong to that stream: an output that the caller drops at once (the norm's
rstd, a prompt's last states, a gradient nobody asked for) would else be given to the
current stream's next allocation while the call still writes it.  They are noted
as used by the current stream as well: one that the caller has read there and freed
must not be given to the call's stream before that reading is done.  On the CPU the
allocations are recorded; on the GPU long work holds a stream up.
"""
import contextlib
import types

import pytest
import torch


@pytest.fixture(scope="module")
def R():
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention
    return retention


def calls(R, dev="cpu"):
    """name -> f(stream): one call of each entry point that allocates outputs."""
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    f32 = lambda *s: torch.randn(*s, generator=g, device=dev)
    b16 = lambda *s: (0.2 * f32(*s)).bfloat16()
    q, k, v, gam = b16(1, 2, 64, 64), b16(1, 2, 64, 64), b16(1, 2, 64, 128), [0.9, 0.95]
    x, w, stat = f32(40, 64), f32(64), f32(40).abs() + 0.5
    X = b16(1, 16, 128)
    W = dict(WQ=b16(128, 128), WK=b16(128, 128), WV=b16(128, 256), WG=b16(128, 256), WO=b16(256, 128))
    shape = dict(H=2, d_k=64, d_v=128, gamma=gam)
    ln, ffn = [f32(128), f32(128)], [b16(128, 256), b16(256, 128)]
    tokens = torch.arange(40, device=dev)
    ids, values = tokens[:, None] % 64, f32(40, 1)
    stats = f32(40, 2)
    s, A, D, bc = f32(2, 70, 32), -f32(32, 16).abs(), f32(32), f32(2, 70, 1, 16)
    h, taps, state = f32(2, 32, 16), f32(32, 4), f32(2, 3, 32)
    S, h2, state2 = f32(1, 2, 64, 128), f32(2, 32, 16), f32(2, 3, 32)  # (states outlive the calls that write them)
    return {
        "chunkwise_fwd": lambda st: R.chunkwise_fwd(q, k, v, gam, stream=st),
        "chunkwise_fwd_noalloc": lambda st: R.chunkwise_fwd_noalloc(q, k, v, gam, stream=st),
        "chunkwise_state": lambda st: R.chunkwise_state(k, v, gam, stream=st),
        "chunkwise_bwd": lambda st: R.chunkwise_bwd(q, k, v, v, gam, stream=st),
        "parallel_fwd": lambda st: R.parallel_fwd(q, k, v, gam, stream=st),
        "recurrent_step": lambda st: R.recurrent_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], S, gam, pos=0, stream=st),
        "rotate": lambda st: R.rotate(q, stream=st),
        "msr_layer_fwd": lambda st: R.msr_layer_fwd(X, **W, **shape, stream=st),
        "retnet_block_fwd": lambda st: R.retnet_block_fwd(X, *ln, *W.values(), *ln, *ffn, **shape, stream=st),
        "gemm_bf16": lambda st: R.gemm_bf16(W["WQ"], W["WV"], stream=st),
        "layernorm_fwd": lambda st: R.layernorm_fwd(x, w, stream=st),
        "layernorm_bwd": lambda st: R.layernorm_bwd(x, x, w, stat, stat, stream=st),
        "token_logprobs": lambda st: R.token_logprobs(x, tokens, top=3, stream=st),
        "distill_fwd": lambda st: R.distill_fwd(x, ids, values, stream=st),
        "distill_bwd": lambda st: R.distill_bwd(x, ids, values, None, stats, stream=st),
        "distill_step": lambda st: R.distill_step(x, ids, values, stream=st),
        "selective_scan_fwd": lambda st: R.selective_scan_fwd(s, s, A, bc, bc, D=D, z=s, stream=st),
        "selective_scan_step": lambda st: R.selective_scan_step(s[:, 0], s[:, 0], A, bc[:, 0], bc[:, 0], h, h_out=h2, stream=st),
        "selective_scan_bwd": lambda st: R.selective_scan_bwd(s, s, A, bc, bc, s, D=D, z=s, dt_bias=D, h_in=h, stream=st),
        "causal_conv_fwd": lambda st: R.causal_conv_fwd(s, taps, D, stream=st),
        "causal_conv_step": lambda st: R.causal_conv_step(s[:, 0], taps, D, state, state_out=state2, stream=st),
        "causal_conv_bwd": lambda st: R.causal_conv_bwd(s, taps, D, s, state_in=state, stream=st),
        "rmsnorm_fwd": lambda st: R.rmsnorm_fwd(x, w, residual=x, stream=st),
        "rmsnorm_quant": lambda st: R.rmsnorm_quant(x, w, residual=x, group=16, stream=st),
        "rmsnorm_bwd": lambda st: R.rmsnorm_bwd(x, x, w, stat, stream=st),
    }


NAMES = ["chunkwise_fwd", "chunkwise_fwd_noalloc", "chunkwise_state", "chunkwise_bwd", "parallel_fwd", "recurrent_step", "rotate",
         "msr_layer_fwd", "retnet_block_fwd", "gemm_bf16", "layernorm_fwd", "layernorm_bwd", "token_logprobs", "distill_fwd",
         "distill_bwd", "distill_step", "selective_scan_fwd", "selective_scan_step", "selective_scan_bwd", "causal_conv_fwd",
         "causal_conv_step", "causal_conv_bwd", "rmsnorm_fwd", "rmsnorm_quant", "rmsnorm_bwd"]


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_allocated_on_the_stream_of_the_call(R, name, monkeypatch):
    make, current, made = calls(R)[name], [None], {}
    side = types.SimpleNamespace(cuda_stream=9)

    def note(real):
        def f(*a, **k):
            t = real(*a, **k)
            made[t.data_ptr()] = current[0]
            return t
        return f

    @contextlib.contextmanager
    def stream_context(s):
        before, current[0] = current[0], s
        try:
            yield
        finally:
            current[0] = before

    class Library:
        def __init__(self, lib):
            self.lib = lib

        def __getattr__(self, n):
            return getattr(self.lib, n) if "workspace_size" in n or "status" in n else (lambda *a: 0)

    for n in ("empty", "zeros", "empty_strided"):
        monkeypatch.setattr(torch, n, note(getattr(torch, n)))
    monkeypatch.setattr(torch.cuda, "stream", stream_context)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, *a, **k: types.SimpleNamespace(cuda_stream=handle))
    monkeypatch.setattr(R, "lib", Library(R.lib))
    monkeypatch.setattr(R, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(R, "_ptrs", lambda *ts: [None if t is None else t.data_ptr() for t in ts])
    out = tensors(make(side))
    mine = [t for t in out if t.data_ptr() in made]
    assert mine and all(s is not None and s.cuda_stream == 9 for s in made.values())


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_dropped_and_freed_outputs(R, name):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    make = calls(R, "cuda")[name]
    torch.cuda.synchronize()
    busy = torch.randn(6144, 6144, device="cuda").bfloat16()
    side = torch.cuda.Stream()

    def hold(stream):
        with torch.cuda.stream(stream):
            for _ in range(8):
                busy @ busy

    for _ in range(2):  # (the first turn leaves freed blocks behind)
        torch.cuda.synchronize()
        sizes = [t.untyped_storage().nbytes() for t in tensors(make(None))]
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        hold(side)
        make(side)  # dropped at once
        filled = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert all(bool((t == 0xA5).all()) for t in filled)
        del filled
    # read on the current stream, late, and freed there at once
    side.wait_stream(torch.cuda.current_stream())
    out = make(side)
    side.synchronize()
    want = [t.clone() for t in tensors(out)]
    torch.cuda.synchronize()
    sizes = [t.untyped_storage().nbytes() for t in tensors(out)]
    hold(torch.cuda.current_stream())
    got = [torch.empty_like(t).copy_(t) for t in tensors(out)]
    del out
    with torch.cuda.stream(side):
        filled = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    del filled


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["chunkwise_bwd", "token_logprobs", "selective_scan_bwd", "rmsnorm_fwd"])
def test_captured_on_a_side_stream(R, name):
    """A call on a stream that joins a capture, some outputs dropped within it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    make = calls(R, "cuda")[name]
    want = [t.clone() for t in tensors(make(None))]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        make(side)
        got = tensors(make(side))
        cur.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in (*got, *copies):
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, c, b in zip(got, copies, want))
    y = make(side)  # eager again
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(tensors(y), want))
