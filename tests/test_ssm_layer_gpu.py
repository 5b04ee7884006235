"""The operators of a selective state space layer as they are used together
(norm with the residual, projections, convolution, scan, the next norm): a
padded batch of prompts and then single tokens, a training step's gradients
against automatic differentiation in 64 bits, and what such programs do around
them: several streams, far strides, graphs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32
DM, E, S, RANK, W = 64, 128, 16, 8, 4


@pytest.fixture(scope="module")
def R():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from linear_recurrent_sequence_gb300 import retention
    return retention


def rand(g, *shape, scale=1.0, dtype=F32):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weights(seed):
    g = gen(seed)
    return dict(norm=1.0 + rand(g, DM, scale=0.1), w_in=rand(g, DM, 2 * E, scale=DM ** -0.5), conv=rand(g, E, W, scale=0.5),
                conv_b=rand(g, E, scale=0.1), w_x=rand(g, E, RANK + 2 * S, scale=E ** -0.5),
                w_dt=rand(g, RANK, E, scale=RANK ** -0.5), dt_bias=rand(g, E, scale=0.5) - 4.0,
                A=-torch.exp(rand(g, E, S, scale=0.5)), D=rand(g, E), w_out=rand(g, E, DM, scale=E ** -0.5),
                norm2=1.0 + rand(g, DM, scale=0.1))


class Layer:
    """One layer on the library's operators; products are torch's."""

    def __init__(self, R, p):
        self.R, self.p = R, p

    def forward(self, x, res, lengths=None, state=None):
        R, p = self.R, self.p
        n, res, rstd = R.rmsnorm_fwd(x, p["norm"], residual=res)
        xz = n @ p["w_in"]
        u, z = xz[..., :E], xz[..., E:]
        conv_in, h_in = (None, None) if state is None else state
        v, conv = R.causal_conv_fwd(u, p["conv"], p["conv_b"], state_in=conv_in, lengths=lengths)
        dbc = v @ p["w_x"]
        dt = dbc[..., :RANK] @ p["w_dt"]
        B, C = dbc[..., RANK:RANK + S], dbc[..., RANK + S:]
        y, h = R.selective_scan_fwd(v, dt, p["A"], B, C, D=p["D"], z=z, dt_bias=p["dt_bias"], h_in=h_in, lengths=lengths)
        out = y @ p["w_out"]
        last, res2, rstd2 = R.rmsnorm_fwd(out, p["norm2"], residual=res)
        self.kept = (n, res, rstd, xz, v, dbc, dt, y, res2, rstd2)
        return last, (conv, h)

    def token(self, x, res, state):
        R, p = self.R, self.p
        conv, h = state
        n, res, _ = R.rmsnorm_fwd(x, p["norm"], residual=res)
        xz = n @ p["w_in"]
        v = R.causal_conv_step(xz[:, :E], p["conv"], p["conv_b"], conv)
        dbc = v @ p["w_x"]
        y = R.selective_scan_step(v, dbc[:, :RANK] @ p["w_dt"], p["A"], dbc[:, RANK:RANK + S], dbc[:, RANK + S:], h, D=p["D"],
                                  z=xz[:, E:], dt_bias=p["dt_bias"])
        return R.rmsnorm_fwd(y @ p["w_out"], p["norm2"], residual=res)[0]

    def backward(self, dlast, dres2):
        """Gradients of the weights, of x and of the residual."""
        R, p = self.R, self.p
        n, res, rstd, xz, v, dbc, dt, y, res2, rstd2 = self.kept
        flat = lambda a, b: a.reshape(-1, a.shape[-1]).t() @ b.reshape(-1, b.shape[-1])
        g = {}
        dout, g["norm2"] = R.rmsnorm_bwd(res2, dlast, p["norm2"], rstd2, dh=dres2)
        g["w_out"], dy = flat(y, dout), dout @ p["w_out"].t()
        B, C = dbc[..., RANK:RANK + S], dbc[..., RANK + S:]
        dxz = torch.empty_like(xz)
        s = R.selective_scan_bwd(v, dt, p["A"], B, C, dy, D=p["D"], z=xz[..., E:], dt_bias=p["dt_bias"], dz=dxz[..., E:])
        g.update(A=s.dA, D=s.dD, dt_bias=s.ddt_bias, w_dt=flat(dbc[..., :RANK], s.ddt))
        ddbc = torch.cat([s.ddt @ p["w_dt"].t(), s.dB, s.dC], -1)
        g["w_x"] = flat(v, ddbc)
        _, g["conv"], g["conv_b"], _ = R.causal_conv_bwd(xz[..., :E], p["conv"], p["conv_b"], s.dx + ddbc @ p["w_x"].t(),
                                                         dx=dxz[..., :E])
        g["w_in"] = flat(n, dxz)
        dx, g["norm"] = R.rmsnorm_bwd(res, dxz @ p["w_in"].t(), p["norm"], rstd, dh=dout)
        return dx, g


def reference(p, x, res):
    """The layer token by token in 64 bits, differentiable."""
    rms = lambda h, w: h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-5) * w
    res = x + res
    xz = rms(res, p["norm"]) @ p["w_in"]
    u, z = xz[..., :E], xz[..., E:]
    pad = torch.cat([torch.zeros_like(u[:, :W - 1]), u], 1)
    N = x.shape[1]
    v = torch.nn.functional.silu(p["conv_b"] + sum(pad[:, k:k + N] * p["conv"][:, k] for k in range(W)))
    dbc = v @ p["w_x"]
    delta = torch.nn.functional.softplus(dbc[..., :RANK] @ p["w_dt"] + p["dt_bias"], threshold=50)
    h, ys = torch.zeros(x.shape[0], E, S, dtype=x.dtype, device=x.device), []
    for t in range(N):
        h = torch.exp(delta[:, t, :, None] * p["A"]) * h + (delta[:, t] * v[:, t])[..., None] * dbc[:, t, None, RANK:RANK + S]
        ys.append((h * dbc[:, t, None, RANK + S:]).sum(-1) + p["D"] * v[:, t])
    out = (torch.stack(ys, 1) * torch.nn.functional.silu(z)) @ p["w_out"]
    return rms(out + res, p["norm2"]), out + res


# Each operator is within about 1e-5 of its sums of magnitudes (its own tests)
# and the fp32 products within K u = 128 x 6e-8 = 8e-6 of theirs; eight of them
# follow one another, each with magnitudes at most about four times the result's
# own: 8 x 4 x 1.5e-5 = 5e-4 of the largest value.
TOL = 5e-4


def near(got, want, what):
    err, top = float((got.double() - want).abs().max()), float(want.abs().max())
    assert err <= TOL * top, f"{what}: {err:.3e} of {top:.3e}"


def test_training_step(R):
    p = weights(1)
    g = gen(2)
    x, res, dlast, dres2 = (rand(g, 2, 70, DM) for _ in range(4))
    layer = Layer(R, p)
    last, _ = layer.forward(x, res)
    dx, grads = layer.backward(dlast, dres2)
    pd = {k: t.double().requires_grad_() for k, t in p.items()}
    xd, rd = x.double().requires_grad_(), res.double().requires_grad_()
    want, res2 = reference(pd, xd, rd)
    near(last, want.detach(), "forward")
    ((want * dlast.double()).sum() + (res2 * dres2.double()).sum()).backward()
    near(dx, xd.grad, "dx")
    near(dx, rd.grad, "dres")
    for k, t in grads.items():
        near(t, pd[k].grad, k)


def test_padded_prompts_then_tokens(R):
    """Three prompts of unequal lengths in one padded call, then five tokens
    each, are the three whole sequences."""
    p = weights(3)
    g = gen(4)
    x, res = rand(g, 3, 45, DM), rand(g, 3, 45, DM)
    lengths = torch.tensor([40, 7, 23], dtype=torch.int32, device="cuda")
    layer = Layer(R, p)
    last, state = layer.forward(x[:, :40].contiguous(), res[:, :40].contiguous(), lengths=lengths)
    rows = torch.arange(3, device="cuda")
    tokens = [layer.token(x[rows, lengths.long() + i], res[rows, lengths.long() + i], state) for i in range(5)]
    pd = {k: t.double() for k, t in p.items()}
    want, _ = reference(pd, x.double(), res.double())
    for i, n in enumerate(lengths.tolist()):
        near(last[i, :n], want[i, :n], f"prompt {i}")
        near(torch.stack([t[i] for t in tokens]), want[i, n:n + 5], f"tokens {i}")


def test_two_streams_at_once(R):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    p = weights(5)
    g = gen(6)
    x, res = rand(g, 2, 3000, DM), rand(g, 2, 3000, DM)
    call = lambda s: (*R.selective_scan_fwd(x, res, p["A"][:DM].contiguous(), x[..., :S], res[..., :S], stream=s),
                      *[t for t in R.selective_scan_bwd(x, res, p["A"][:DM].contiguous(), x[..., :S], res[..., :S], res, stream=s)
                        if t is not None],
                      *R.causal_conv_bwd(x, p["conv"][:DM].contiguous(), None, res, stream=s)[:2],
                      *R.rmsnorm_bwd(x, res, None, want_rstd, stream=s))
    _, _, want_rstd = R.rmsnorm_fwd(x)
    want = call(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [call(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_far_strides(R):
    """Tokens whose offsets pass 2^31 elements."""
    g = gen(7)
    step = (1 << 30) + 16
    buf = torch.zeros(3 * step + 64, dtype=torch.bfloat16, device="cuda")
    far = buf.as_strided((1, 4, 16), (4 * step, step, 1), 16)
    near_x = rand(g, 1, 4, 16, dtype=torch.bfloat16)
    far.copy_(near_x)
    A, w = -torch.rand(16, 4, generator=g, device="cuda"), rand(g, 16, 4)
    dt, B, dy = rand(g, 1, 4, 16, dtype=torch.bfloat16), rand(g, 1, 4, 4, dtype=torch.bfloat16), rand(g, 1, 4, 16, dtype=torch.bfloat16)
    for a, b in zip(R.selective_scan_fwd(far, dt, A, B, B, z=far), R.selective_scan_fwd(near_x, dt, A, B, B, z=near_x)):
        assert torch.equal(a, b)
    for a, b in zip(R.selective_scan_bwd(far, dt, A, B, B, far, z=far), R.selective_scan_bwd(near_x, dt, A, B, B, near_x, z=near_x)):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(R.causal_conv_fwd(far, w)[0], R.causal_conv_fwd(near_x, w)[0])
    assert torch.equal(R.causal_conv_bwd(far, w, None, dy)[0], R.causal_conv_bwd(near_x, w, None, dy)[0])
    assert torch.equal(R.rmsnorm_fwd(far)[0], R.rmsnorm_fwd(near_x)[0])
    want = R.selective_scan_fwd(near_x, dt, A, B, B)[0]
    assert torch.equal(R.selective_scan_fwd(near_x, dt, A, B, B, out=far)[0], want)


def test_decode_steps_in_a_graph(R):
    """Tokens through a captured step: the states move on with each replay."""
    p = weights(8)
    g = gen(9)
    x, res = rand(g, 2, 12, DM), rand(g, 2, 12, DM)
    layer = Layer(R, p)
    state = (torch.zeros(2, W - 1, E, device="cuda"), torch.zeros(2, E, S, device="cuda"))
    xin, rin = x[:, 0].clone(), res[:, 0].clone()
    layer.token(xin, rin, (state[0].clone(), state[1].clone()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.token(xin, rin, state)
    for t in state:
        t.zero_()
    got = []
    for t in range(12):
        xin.copy_(x[:, t])
        rin.copy_(res[:, t])
        graph.replay()
        got.append(out.clone())
    want, _ = reference({k: t.double() for k, t in p.items()}, x.double(), res.double())
    near(torch.stack(got, 1), want, "tokens")
