"""Host-side checks of what the binding hands to the LayerNorm, logits and
distillation entry points; the library is replaced by a recorder, no GPU
needed."""
import ctypes

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """(the binding, the descriptors that its calls handed to the library)."""
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention as R
    given = []

    class Library:
        def __init__(self, lib):
            self.lib = lib

        def __getattr__(self, name):
            if "workspace_size" in name or "status" in name:
                return getattr(self.lib, name)

            def call(desc, *args):
                d = desc._obj
                given.append(type(d).from_buffer_copy(ctypes.string_at(ctypes.addressof(d), ctypes.sizeof(d))))
                return 0
            return call

    monkeypatch.setattr(R, "lib", Library(R.lib))
    monkeypatch.setattr(R, "_ptrs", lambda *ts: [None if t is None else t.data_ptr() for t in ts])
    monkeypatch.setattr(R, "_stream", lambda s: None)
    yield R, given
    R._ln_desc.cache_clear()  # (sizes and descriptors of the stand-in)
    R._logits_desc.cache_clear()


def test_options_as_tensors_are_read_at_each_call(calls):
    """A temperature or an epsilon that a program keeps in a tensor and moves
    in place (an annealing schedule)."""
    R, given = calls
    x, ids, values = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2)
    t = torch.tensor(1.0)
    stats = torch.zeros(3, 2)
    for f in (lambda: R.token_logprobs(x, temperature=t), lambda: R.distill_fwd(x, ids, values, temperature=t),
              lambda: R.distill_bwd(x, ids, values, None, stats, temperature=t),
              lambda: R.distill_step(x, ids, values, temperature=t)):
        for want in (1.0, 4.0, 0.25):
            t.fill_(want)
            f()
            assert given[-1].temperature == want
    eps = torch.tensor(0.5)
    for want in (0.5, 0.125):
        eps.fill_(want)
        R.layernorm_fwd(x, eps=eps)
        assert given[-1].eps == want
    top = torch.tensor(2)
    for want in (2, 3):
        top.fill_(want)
        out = R.token_logprobs(x, top=top)
        assert given[-1].top == want and out[3].shape == (3, want)
    with pytest.raises(TypeError):
        R.token_logprobs(x, top=2.5)


def test_workspace_size_is_that_of_the_device(calls, monkeypatch):
    """layernorm_bwd's workspace depends on the device's SMs: tensors of equal
    shapes on two unlike devices (here the host and torch's meta device) get
    each its own."""
    R, given = calls
    sizes = {"cpu": 4096, "meta": 8192}
    made, real = [], torch.empty
    now = []
    lib = R.lib
    lib.__dict__["retnet_layernorm_bwd_workspace_size"] = lambda d: sizes[now[-1]]

    def empty(*a, **k):
        if k.get("dtype") is torch.uint8:
            made.append((a[0], str(k["device"])))
        return real(*a, **k)

    monkeypatch.setattr(torch, "empty", empty)
    for dev in ("cpu", "meta", "cpu"):
        now.append(dev)
        x, stat = torch.zeros(5, 72, device=dev), torch.zeros(5, device=dev)
        R.layernorm_bwd(x, x, None, stat, stat)
        assert made[-1] == (sizes[dev], dev)
