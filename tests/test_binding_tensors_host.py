"""Host-side check that every tensor of a decode step passes the binding's
check for CUDA tensors on the current device before its address reaches the
library (a host address would reach a kernel); no GPU needed."""
import torch


def test_decode_step_checks_weights_and_states(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    from linear_recurrent_sequence_gb300 import retention as R
    checked = set()

    def ptr(t):
        checked.add(t.data_ptr())
        return t.data_ptr()

    class Library:
        def __getattr__(self, name):
            return (lambda *a: 512) if "workspace_size" in name else (lambda *a: 0)

    monkeypatch.setattr(R, "lib", Library())
    monkeypatch.setattr(R, "_ptr", lambda t: None if t is None else ptr(t))
    monkeypatch.setattr(R, "_ptrs", lambda *ts: [None if t is None else ptr(t) for t in ts])
    monkeypatch.setattr(R, "_stream", lambda s: None)
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    layers = [dict(ln1_w=torch.zeros(64), ln1_b=torch.zeros(64), WQ=b16(64, 64), WK=b16(64, 64), WV=b16(64, 64),
                   WG=b16(64, 64), WO=b16(64, 64), ln2_w=torch.zeros(64), ln2_b=torch.zeros(64), W1=b16(64, 128),
                   W2=b16(128, 64)) for _ in range(2)]
    X = b16(3, 64)
    S, z = ([torch.zeros(3, 1, 64, d) for _ in layers] for d in (64, 1))
    R.retnet_decode_step(X, layers, S, z, H=1, d_k=64, d_v=64, gamma=[0.9], pos=0)
    given = [X, *S, *z, *(t for L in layers for t in L.values())]
    assert all(t.data_ptr() in checked for t in given)
