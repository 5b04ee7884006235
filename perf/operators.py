"""The operators around a RetNet stack's output: what is timed, and on which sizes.

Three operators, each direction of them a case kind of its own:

  layernorm_fwd / layernorm_bwd   the final (and every block's) LayerNorm with the statistics it
                                  saves, and its gradients with the sums of dw and db over the rows;
  logprobs                        log probabilities of given tokens, entropy and top alternatives
                                  of the output head's logits;
  distill_fwd / _bwd / _step      the distillation loss against a teacher's top logits, its gradient
                                  with respect to the student's logits, and both in one call.

``own`` false: plain torch operations in 32 bits.  ``own`` true: the framework's entry points.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
ELEM = {BF16: 2, F32: 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step's final LayerNorm at batch 8 of the 6.7B-scale width: latency.
        dict(name="ln fwd decode", op="layernorm_fwd", n0=1, n1=8, d=4096, dtype=BF16, pad=0),
        # LayerNorm over two 8192-token sequences of the same width: bandwidth.
        dict(name="ln fwd tokens", op="layernorm_fwd", n0=2, n1=8192, d=4096, dtype=BF16, pad=0),
        # An odd width read out of a wider buffer (rows not aligned), fp32.
        dict(name="ln fwd odd f32", op="layernorm_fwd", n0=3, n1=1001, d=1537, dtype=F32, pad=3),
        # A training step's LayerNorm gradients: 8192 tokens of the 6.7B-scale width.
        dict(name="ln bwd tokens", op="layernorm_bwd", n0=1, n1=8192, d=4096, dtype=BF16, pad=0),
        # The same in fp32 at an odd width.
        dict(name="ln bwd odd f32", op="layernorm_bwd", n0=1, n1=2053, d=1537, dtype=F32, pad=0),
        # Serving: log probability of the sampled token and 20 alternatives, batch 8, large vocabulary.
        dict(name="logprobs decode", op="logprobs", n0=1, n1=8, V=131072, dtype=BF16, top=20,
             temperature=1.0, shift=0, masked=0.0),
        # Scoring two prompts of 2048 tokens: every position but the last against the next token.
        dict(name="logprobs prompt", op="logprobs", n0=2, n1=2048, V=65536, dtype=BF16, top=5,
             temperature=1.0, shift=1, masked=0.0),
        # A teacher's 128 top alternatives in fp32 at an odd vocabulary with masked tokens.
        dict(name="logprobs top f32", op="logprobs", n0=1, n1=301, V=50001, dtype=F32, top=128,
             temperature=2.0, shift=0, masked=0.3),
        # Distillation loss of an evaluation batch (no gradient).
        dict(name="distill fwd", op="distill_fwd", n0=1, n1=1024, V=65536, dtype=BF16, top=64,
             temperature=2.0, tail=False),
        # The gradient from saved statistics, fp32, odd vocabulary, with the rest bucket.
        dict(name="distill bwd f32", op="distill_bwd", n0=1, n1=257, V=50001, dtype=F32, top=20,
             temperature=1.0, tail=True),
        # A training step's loss and gradient in one call: 4096 tokens.
        dict(name="distill step", op="distill_step", n0=2, n1=2048, V=65536, dtype=BF16, top=64,
             temperature=2.0, tail=False),
        # The same for a handful of tokens with the rest bucket.
        dict(name="distill step few", op="distill_step", n0=1, n1=8, V=32768, dtype=BF16, top=16,
             temperature=1.0, tail=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm_fwd", "layernorm_bwd", "logprobs", "distill_fwd", "distill_bwd",
                     "distill_step"])
    dtype = rng.choice([BF16, F32])
    if op.startswith("layernorm"):
        d = _log_int(rng, 64, 16384)
        d = d // 8 * 8 if rng.random() < 0.6 else d
        most = (1 << 28) // (d * ELEM[dtype] * 3)
        n1 = _log_int(rng, 1, min(most, 32768))
        return dict(op=op, n0=1, n1=n1, d=d, dtype=dtype, pad=rng.choice([0, 0, 0, 8, 3]))
    V = _log_int(rng, 1000, 160000)
    V = V // 64 * 64 if rng.random() < 0.5 else V
    most = (1 << 29) // (V * ELEM[dtype])
    n0, n1 = rng.choice([1, 1, 2]), _log_int(rng, 1 if op == "logprobs" else 4, min(most // 2, 4096))
    top = _log_int(rng, 1, 128)
    if op == "logprobs":
        return dict(op=op, n0=n0, n1=n1, V=V, dtype=dtype, top=rng.choice([0, top]),
                    temperature=rng.choice([1.0, 0.7, 2.0]), shift=rng.choice([0, 1]),
                    masked=rng.choice([0.0, 0.0, 0.3]))
    return dict(op=op, n0=n0, n1=n1, V=V, dtype=dtype, top=top, temperature=rng.choice([1.0, 2.0]),
                tail=rng.choice([False, True]))


def work(case):
    rows, e, op = case["n0"] * case["n1"], ELEM[case["dtype"]], case["op"]
    if op == "layernorm_fwd":
        # x read, y written; the gain and bias once; mean and rstd written
        return dict(bytes=rows * case["d"] * 2 * e + case["d"] * 8 + rows * 8,
                    flops=rows * case["d"] * 7)
    if op == "layernorm_bwd":
        # x and dy read, dx written; the gain read, dw and db written; mean and rstd read
        return dict(bytes=rows * case["d"] * 3 * e + case["d"] * 12 + rows * 8,
                    flops=rows * case["d"] * 13)
    n, k = rows * case["V"], case["top"]
    if op == "logprobs":
        # the logits once; a token, two results and k (id, value) pairs a row
        return dict(bytes=n * e + rows * (16 + 12 * k), flops=n * 7)
    if op == "distill_fwd":
        return dict(bytes=n * e + rows * (12 * k + 12), flops=n * 5)
    # the logits read and their gradient written
    return dict(bytes=n * 2 * e + rows * (12 * k + 16), flops=n * (5 if op == "distill_bwd" else 10))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _padded(n0, n1, d, pad, dtype, fill):
    """A [n0, n1, d] view of a buffer whose rows are d + pad wide."""
    buf = torch.empty(n0, n1, d + pad, dtype=dtype, device="cuda")
    view = buf[..., :d]
    view.copy_(fill)
    return view


def _prepare_layernorm(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n0, n1, d = case["n0"], case["n1"], case["d"]
    x = torch.randn(n0, n1, d, generator=g, device="cuda")
    # a level of its own for each row and for each channel, as a residual stream has
    x += 0.5 * torch.randn(n0, n1, 1, generator=g, device="cuda")
    x *= 1.0 + torch.rand(d, generator=g, device="cuda")
    st = dict(case=dict(case), eps=1e-5,
              x=_padded(n0, n1, d, case["pad"], dt, x),
              w=1.0 + 0.1 * torch.randn(d, generator=g, device="cuda"),
              b=0.1 * torch.randn(d, generator=g, device="cuda"))
    if case["op"] == "layernorm_fwd":
        st["y"] = torch.empty(n0, n1, d, dtype=dt, device="cuda")
        st["mean"] = torch.empty(n0, n1, dtype=torch.float32, device="cuda")
        st["rstd"] = torch.empty(n0, n1, dtype=torch.float32, device="cuda")
        return st
    xd = st["x"].double()
    st["mean"] = xd.mean(-1).float()
    st["rstd"] = (xd.var(-1, unbiased=False) + st["eps"]).rsqrt().float()
    dy = 0.05 * torch.randn(n0, n1, d, generator=g, device="cuda")
    st["dy"] = _padded(n0, n1, d, case["pad"], dt, dy)
    st["dx"] = torch.empty(n0, n1, d, dtype=dt, device="cuda")
    st["dw"] = torch.empty(d, device="cuda")
    st["db"] = torch.empty(d, device="cuda")
    return st


def _logits(case, g, n1):
    """Logits with a few strong tokens a row, as an output head gives them."""
    n0, V = case["n0"], case["V"]
    x = 2.0 * torch.randn(n0, n1, V, generator=g, device="cuda")
    strong = torch.randint(0, V, (n0, n1, 4), generator=g, device="cuda")
    x.scatter_add_(2, strong, 6.0 * torch.rand(n0, n1, 4, generator=g, device="cuda") + 4.0)
    return x, strong


def _prepare_logprobs(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n0, n1, V, k = case["n0"], case["n1"], case["V"], case["top"]
    x, strong = _logits(case, g, n1 + case["shift"])
    tokens = strong[:, case["shift"]:, 0].clone() if case["shift"] else strong[..., 0].clone()
    if case["masked"] > 0.0:
        # tokens that a grammar rules out, the scored ones never among them
        drop = torch.rand(n0, n1 + case["shift"], V, generator=g, device="cuda") < case["masked"]
        drop.scatter_(2, strong, False)
        x.masked_fill_(drop, -math.inf)
        del drop
    # positions without a token to score (padding)
    none = torch.rand(n0, n1, generator=g, device="cuda") < 0.02
    tokens = torch.where(none, torch.full_like(tokens, -100), tokens)
    logits = x.to(dt)
    if case["shift"]:
        logits = logits[:, :-1]
    st = dict(case=dict(case), logits=logits, tokens=tokens,
              logprob=torch.empty(n0, n1, device="cuda"), entropy=torch.empty(n0, n1, device="cuda"),
              top_logprobs=None, top_ids=None)
    if k:
        st["top_logprobs"] = torch.empty(n0, n1, k, device="cuda")
        st["top_ids"] = torch.empty(n0, n1, k, dtype=torch.int64, device="cuda")
    return st


def _prepare_distill(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n0, n1, V, k, T = case["n0"], case["n1"], case["V"], case["top"], case["temperature"]
    x, _ = _logits(case, g, n1)
    # the teacher: the student's logits and a difference of its own
    t = x + torch.randn(n0, n1, V, generator=g, device="cuda")
    student = x.to(dt)
    del x
    values, ids = t.topk(k, dim=-1)
    if case["tail"]:  # log probabilities of the whole vocabulary
        values = values / T - torch.logsumexp(t / T, -1, keepdim=True)
    del t
    rows = n0 * n1
    weight = torch.full((n0, n1), 1.0 / rows, device="cuda")
    weight *= (torch.rand(n0, n1, generator=g, device="cuda") > 0.02)  # padding has no weight
    if rows > 4 and k > 1:  # a shorter list in some rows
        short = torch.rand(n0, n1, generator=g, device="cuda") < 0.05
        ids[..., k - 1] = torch.where(short, torch.full_like(ids[..., 0], -1), ids[..., k - 1])
    st = dict(case=dict(case), student=student, ids=ids.contiguous(), values=values.contiguous(),
              weight=weight, loss=torch.empty(n0, n1, device="cuda"),
              stats=torch.empty(n0, n1, 2, device="cuda"), dstudent=None)
    if case["op"] == "distill_bwd":
        st["stats"] = _plain_stats(student, st["ids"], T)
    if case["op"] != "distill_fwd":
        st["dstudent"] = torch.empty(n0, n1, V, dtype=dt, device="cuda")
    return st


def _plain_stats(student, ids, T):
    """The forward's saved logsumexp of student / T: over the vocabulary, and without the ids."""
    s = student.double() / T
    lse = torch.logsumexp(s, -1)
    return torch.stack([lse, torch.logsumexp(s.masked_fill_(_listed_ids(ids, s.shape[-1]), -math.inf), -1)],
                       -1).float()


def _listed_ids(ids, V):
    """[.., V] truth values: the token is among the row's ids (negative ids are absent)."""
    hit = torch.zeros(*ids.shape[:-1], V + 1, dtype=torch.bool, device=ids.device)
    return hit.scatter_(-1, torch.where(ids < 0, V, ids), True)[..., :V]


def prepare(case, seed):
    if case["op"].startswith("layernorm"):
        return _prepare_layernorm(case, seed)
    return (_prepare_logprobs if case["op"] == "logprobs" else _prepare_distill)(case, seed)


# ------------------------------------------------------------------ plain forms
def _plain_layernorm_fwd(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    c = x - mean
    rstd = torch.rsqrt((c * c).mean(-1, keepdim=True) + st["eps"])
    y = c * rstd * st["w"] + st["b"]
    return dict(y=y.to(st["x"].dtype), mean=mean[..., 0], rstd=rstd[..., 0])


def _plain_layernorm_bwd(st):
    x, dy, rstd = st["x"].float(), st["dy"].float(), st["rstd"][..., None]
    xhat = (x - st["mean"][..., None]) * rstd
    gw = dy * st["w"]
    dx = rstd * (gw - gw.mean(-1, keepdim=True) - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dict(dx=dx.to(st["x"].dtype), dw=(dy * xhat).sum((0, 1)), db=dy.sum((0, 1)))


def _ordered_keys(x):
    """int64 keys of fp32 values [.., V]: by value, equal values by the lower index first."""
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    return order * (1 << 32) + torch.arange(x.shape[-1] - 1, -1, -1, device=x.device)


def _plain_logprobs(st):
    case, x = st["case"], st["logits"].float()
    T, k, V = case["temperature"], case["top"], case["V"]
    s = x / T
    top = s.amax(-1, keepdim=True)
    y = s - top
    e = torch.exp(y)
    z = e.sum(-1, keepdim=True)
    logz = torch.log(z)
    entropy = logz - (torch.where(e > 0, y * e, 0.0)).sum(-1, keepdim=True) / z
    tokens = st["tokens"]
    lp = y.gather(-1, tokens.clamp(min=0)[..., None]) - logz
    out = dict(logprob=torch.where(tokens < 0, 0.0, lp[..., 0]), entropy=entropy[..., 0])
    if k:
        ids = (V - 1) - (_ordered_keys(x).topk(k, dim=-1).values & 0xFFFFFFFF)
        out["top_logprobs"] = y.gather(-1, ids) - logz
        out["top_ids"] = torch.where(torch.isinf(out["top_logprobs"]), -1, ids)
    return out


def _plain_teacher(st):
    """The teacher's probabilities of its ids (0 where absent) and of the rest."""
    T, ids = st["case"]["temperature"], st["ids"]
    if st["case"]["tail"]:
        p = torch.where(ids < 0, 0.0, torch.exp(st["values"]))
        return p, (1.0 - p.sum(-1)).clamp(min=0.0)
    v = torch.where(ids < 0, -math.inf, st["values"] / T)
    e = torch.exp(v - v.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True), None


def _term(p, logp, logq):
    """p log(p / q) - p + q, never negative: over all buckets these add up to sum p log(p / q)."""
    delta = logp - logq
    return torch.where(p > 0, p * (delta + torch.expm1(-delta)), torch.exp(logq))


def _plain_loss(st, s, p, rest):
    """Loss of each row and its saved statistics, from s = student / T in 32 bits."""
    T, ids = st["case"]["temperature"], st["ids"]
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top)
    lse = torch.log(e.sum(-1)) + top[..., 0]
    lse_rest = torch.log(e.masked_fill(_listed_ids(ids, s.shape[-1]), 0.0).sum(-1)) + top[..., 0]
    logq = torch.where(ids < 0, -math.inf, s.gather(-1, ids.clamp(min=0)) - lse[..., None])
    if rest is None:  # no bucket of the teacher's: what the student gives the rest is lost
        bucket = torch.exp(lse_rest - lse)
    else:
        bucket = _term(rest, torch.log(rest), lse_rest - lse)
    loss = _term(p, torch.log(p), logq).sum(-1) + bucket
    return T * T * loss, torch.stack([lse, lse_rest], -1)


def _plain_gradient(st, s, p, rest, stats):
    T, ids = st["case"]["temperature"], st["ids"]
    grad = torch.exp(s - stats[..., :1])
    if rest is not None:
        other = rest[..., None] * torch.exp(s - stats[..., 1:])
        grad = grad - torch.where(_listed_ids(ids, s.shape[-1]), 0.0, other)
    grad.scatter_add_(-1, ids.clamp(min=0), -p)
    grad *= T * st["weight"][..., None]
    return grad.to(st["student"].dtype)


def _plain_distill(st):
    case = st["case"]
    s = st["student"].float() / case["temperature"]
    p, rest = _plain_teacher(st)
    if case["op"] == "distill_bwd":
        return dict(dstudent=_plain_gradient(st, s, p, rest, st["stats"]))
    loss, stats = _plain_loss(st, s, p, rest)
    if case["op"] == "distill_fwd":
        return _forward_outputs(case, loss, stats)
    return dict(loss=loss, dstudent=_plain_gradient(st, s, p, rest, stats))


def _forward_outputs(case, loss, stats):
    """The loss and what the backward needs: the rest's logsumexp only with the rest bucket."""
    out = dict(loss=loss, lse=stats[..., 0])
    if case["tail"]:
        out["lse_rest"] = stats[..., 1]
    return out


# ------------------------------------------------------------------ one pass
def _run_own(st):
    from linear_recurrent_sequence_gb300 import retention as R
    case = st["case"]
    op = case["op"]
    if op == "layernorm_fwd":
        y, mean, rstd = R.layernorm_fwd(st["x"], st["w"], st["b"], eps=st["eps"], out=st["y"],
                                        mean=st["mean"], rstd=st["rstd"])
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "layernorm_bwd":
        dx, dw, db = R.layernorm_bwd(st["x"], st["dy"], st["w"], st["mean"], st["rstd"],
                                     dx=st["dx"], dw=st["dw"], db=st["db"])
        return dict(dx=dx, dw=dw, db=db)
    if op == "logprobs":
        lp, ent, top_lp, top_ids = R.token_logprobs(
            st["logits"], st["tokens"], top=case["top"], temperature=case["temperature"],
            logprob=st["logprob"], entropy=st["entropy"], top_logprobs=st["top_logprobs"],
            top_ids=st["top_ids"])
        out = dict(logprob=lp, entropy=ent)
        if case["top"]:
            out.update(top_logprobs=top_lp, top_ids=top_ids)
        return out
    kw = dict(temperature=case["temperature"], tail=case["tail"])
    if op == "distill_fwd":
        loss, stats = R.distill_fwd(st["student"], st["ids"], st["values"], loss=st["loss"],
                                    stats=st["stats"], **kw)
        return _forward_outputs(case, loss, stats)
    if op == "distill_bwd":
        return dict(dstudent=R.distill_bwd(st["student"], st["ids"], st["values"], st["weight"],
                                           st["stats"], dstudent=st["dstudent"], **kw))
    loss, grad = R.distill_step(st["student"], st["ids"], st["values"], st["weight"],
                                loss=st["loss"], dstudent=st["dstudent"], **kw)
    return dict(loss=loss, dstudent=grad)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "layernorm_fwd":
        return _plain_layernorm_fwd(state)
    if op == "layernorm_bwd":
        return _plain_layernorm_bwd(state)
    return _plain_logprobs(state) if op == "logprobs" else _plain_distill(state)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "layernorm_fwd":
        x = st["x"].double()
        var, mean = torch.var_mean(x, -1, unbiased=False)
        rstd = 1.0 / torch.sqrt(var + st["eps"])
        y = (x - mean[..., None]) * rstd[..., None] * st["w"].double() + st["b"].double()
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "layernorm_bwd":
        d = case["d"]
        x, dy = st["x"].double().reshape(-1, d), st["dy"].double().reshape(-1, d)
        m, r = st["mean"].double().reshape(-1, 1), st["rstd"].double().reshape(-1, 1)
        h = (x - m) * r
        a = dy * st["w"].double()
        c1, c2 = a.sum(1, keepdim=True) / d, (a * h).sum(1, keepdim=True) / d
        return dict(dx=((a - c1 - h * c2) * r).reshape(st["x"].shape), dw=(dy * h).sum(0),
                    db=dy.sum(0))
    T, V, rows = float(case["temperature"]), case["V"], case["n0"] * case["n1"]
    block = max(1, (1 << 26) // V)
    parts = []
    if op == "logprobs":
        x2, t2 = st["logits"].reshape(rows, V), st["tokens"].reshape(rows)
        for i in range(0, rows, block):
            lp = torch.log_softmax(x2[i:i + block].double() / T, -1)
            prob = lp.exp()
            t = t2[i:i + block]
            one = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
            got = [one, -torch.nan_to_num(prob * lp, nan=0.0).sum(1)]
            if case["top"]:
                got.append(lp.topk(case["top"], 1).values)
            parts.append(got)
        out = [torch.cat(c).reshape(case["n0"], case["n1"], *c[0].shape[1:]) for c in zip(*parts)]
        res = dict(logprob=out[0], entropy=out[1])
        if case["top"]:
            res.update(top_logprobs=out[2], top_ids=None)
        return res
    k = case["top"]
    x2, id2, v2 = (st[n].reshape(rows, -1) for n in ("student", "ids", "values"))
    w2, stats2 = st["weight"].reshape(rows), st["stats"].reshape(rows, 2)
    for i in range(0, rows, block):
        ids, v = id2[i:i + block], v2[i:i + block].double()
        there = ids >= 0
        safe = torch.where(there, ids, 0)
        s = x2[i:i + block].double() / T
        lse = torch.logsumexp(s, 1)
        p = torch.where(there, v.exp() if case["tail"] else
                        torch.softmax(torch.where(there, v / T, -math.inf), 1), 0.0)
        dense = torch.zeros_like(s).scatter_add_(1, safe, p)
        inside = torch.zeros_like(s).scatter_add_(1, safe, there.double()) > 0
        lse_rest = torch.logsumexp(s.masked_fill(inside, -math.inf), 1)
        loss = (torch.special.xlogy(p, p) - p * (s.gather(1, safe) - lse[:, None])).sum(1)
        pr = (1.0 - p.sum(1)).clamp(min=0.0)
        if case["tail"]:
            loss = loss + torch.special.xlogy(pr, pr) - pr * (lse_rest - lse)
        if op == "distill_fwd":
            parts.append([T * T * loss, lse, lse_rest])
            continue
        if op == "distill_bwd":
            lse, lse_rest = stats2[i:i + block, 0].double(), stats2[i:i + block, 1].double()
        grad = (s - lse[:, None]).exp() - dense
        if case["tail"]:
            grad -= torch.where(inside, 0.0, pr[:, None] * (s - lse_rest[:, None]).exp())
        grad *= T * w2[i:i + block, None].double()
        # rounded once to the gradient's type, to hold a whole batch of them
        parts.append([T * T * loss, grad.to(torch.float32)])
    shape = (case["n0"], case["n1"])
    out = [torch.cat(c) for c in zip(*parts)]
    out = [o.reshape(*shape, *o.shape[1:]) for o in out]
    if op == "distill_fwd":
        res = dict(loss=out[0], lse=out[1])
        if case["tail"]:
            res["lse_rest"] = out[2]
        return res
    if op == "distill_bwd":
        return dict(dstudent=out[1])
    return dict(loss=out[0], dstudent=out[1])
