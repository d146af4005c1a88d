"""Cases for the operators on [rows, vocab] logits beside the sampling step: the step with min-p, the top
logits of a row with their log-sum-exps, and the distillation loss from a teacher's top logits with its gradient.

Where `own` is false, `run` computes them in plain torch operations; where it is true it calls
decode_token_sampling_gb300.
"""

import math

import torch

own = False

BIG_V = 151936


def listed():
    return [
        # min-p sampling: one sequence decoding; a bf16 serving batch with every stage in use; a large fp32 batch
        # with the repetition penalty, a third of the rows on min-p alone
        dict(name="minp one row", op="sample", B=1, V=32000, dtype="f32", mix="minp", seen=0),
        dict(name="minp batch bf16", op="sample", B=64, V=128256, dtype="bf16", mix="all", seen=0),
        dict(name="minp large penalty", op="sample", B=256, V=BIG_V, dtype="f32", mix="all", seen=512),
        # top logits: log-probabilities for one sequence, for a serving batch, a long list over an odd vocabulary
        # in a padded buffer, and a teacher's pass over a batch of training tokens
        dict(name="top one row", op="top", B=1, V=BIG_V, ld=BIG_V, n=20, dtype="f32", tau=1.0),
        dict(name="top serving batch", op="top", B=256, V=BIG_V, ld=BIG_V, n=20, dtype="bf16", tau=1.0),
        dict(name="top long list odd", op="top", B=96, V=50001, ld=50048, n=1000, dtype="f32", tau=0.7),
        dict(name="top teacher pass", op="top", B=2048, V=BIG_V, ld=BIG_V, n=64, dtype="bf16", tau=2.0),
        # distillation: a small evaluation, an evaluation over a training batch, a loss with its gradient over
        # odd rows and over a training batch (a quarter of whose tokens carry no loss), and the autograd pair
        dict(name="distill loss small", op="loss", N=16, V=32000, ld=32000, K=16, dtype="f32", tau=1.0, rest=False, masked=0),
        dict(name="distill loss batch", op="loss", N=4096, V=BIG_V, ld=BIG_V, K=64, dtype="bf16", tau=2.0, rest=True, masked=1024),
        dict(name="distill step odd", op="step", N=130, V=50001, ld=50001, K=100, dtype="f32", tau=1.5, rest=True, masked=30),
        dict(name="distill step batch", op="step", N=4096, V=BIG_V, ld=BIG_V, K=64, dtype="bf16", tau=2.0, rest=True, masked=1024),
        dict(name="distill autograd", op="autograd", N=1024, V=128256, ld=128256, K=32, dtype="bf16", tau=1.0, rest=False, masked=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "top", "loss", "step", "autograd"])
    V = _log(rng, 1000, BIG_V)
    dtype = rng.choice(["f32", "bf16"])
    if op == "sample":
        return dict(op=op, B=_log(rng, 1, 256), V=V, dtype=dtype, mix=rng.choice(["all", "minp"]), seen=rng.choice([0, 100, 512]))
    ld = rng.choice([V, -(-V // 64) * 64])
    tau = rng.choice([0.7, 1.0, 2.0])
    if op == "top":
        return dict(op=op, B=_log(rng, 1, 1024), V=V, ld=ld, n=_log(rng, 1, min(V, 1024)), dtype=dtype, tau=tau)
    N = _log(rng, 1, 2048)
    return dict(op=op, N=N, V=V, ld=ld, K=_log(rng, 1, 512), dtype=dtype, tau=tau, rest=rng.random() < 0.5, masked=N // 4)


# ---- inputs ------------------------------------------------------------------------------------------

def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _logits(g, N, V, ld, sigma, bonus):
    """N(0, sigma) plus bonus / sqrt(r) for a rank r drawn per token; the columns behind V hold junk."""
    x = torch.randn(N, ld, device="cuda", generator=g).mul_(sigma)
    r = torch.rand(N, ld, device="cuda", generator=g).mul_(V).add_(1.0)
    x.addcmul_(r.rsqrt_(), torch.full((), bonus, device="cuda"))
    return x


def _prepare_sample(case, g):
    B, V = case["B"], case["V"]
    u = lambda lo, hi: torch.rand(B, device="cuda", generator=g) * (hi - lo) + lo  # noqa: E731
    s = dict(case=case, logits=_logits(g, B, V, V, 2.5, 10.0).to(_dt(case)), temperature=u(0.5, 1.2), min_p=u(0.02, 0.2))
    kind = torch.arange(B, device="cuda") % 3 if case["mix"] == "all" else torch.full((B,), 2, device="cuda")
    k = torch.randint(1, min(1024, V) + 1, (B,), device="cuda", generator=g)
    s["top_k"] = torch.where(kind == 0, k, torch.zeros_like(k)).to(torch.int32)  # 0: the stage is off
    s["top_p"] = torch.where(kind == 2, torch.ones(B, device="cuda"), u(0.5, 0.99))
    s["q"] = torch.empty(B, V, device="cuda").exponential_(generator=g)
    s["workspace"] = torch.zeros(256 + 32896 * min(B, 1024), dtype=torch.uint8, device="cuda")
    if case["seen"]:
        n = case["seen"]
        s["seen_ids"] = torch.randint(0, V, (B * n,), device="cuda", generator=g, dtype=torch.int32)
        s["seen_indptr"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
        s["penalty"] = u(1.05, 1.3)
    return s


def _prepare_top(case, g):
    B, V = case["B"], case["V"]
    x = _logits(g, B, V, case["ld"], 2.5, 10.0).to(_dt(case))[:, :V]
    return dict(case=case, logits=x, tokens=torch.randint(0, V, (B,), device="cuda", generator=g))


def _prepare_distill(case, g):
    """A student that is its teacher with noise, the top tokens holding most of the mass; the teacher's lists are
    ragged: one row in four is shorter."""
    N, V, K, tau = case["N"], case["V"], case["K"], case["tau"]
    t = _logits(g, N, V, case["ld"], 2.0, 30.0)
    student = torch.empty_like(t, dtype=_dt(case))
    student.copy_(torch.randn(N, case["ld"], device="cuda", generator=g).add_(t))
    t = t[:, :V]
    values, ids = t.topk(K, dim=1)
    ids = ids.to(torch.int32)
    s = dict(case=case, student=student[:, :V], values=values.to(_dt(case)), rest=None)
    if case["rest"]:
        t.scatter_(1, ids.long(), -math.inf)
        s["rest"] = t.div_(tau).logsumexp(1)
    short = (torch.arange(N, device="cuda") % 4 == 1)[:, None] & (torch.arange(K, device="cuda") >= (K + 1) // 2)[None, :]
    s["ids"] = torch.where(short, torch.full_like(ids, -1), ids)
    weight = torch.rand(N, device="cuda", generator=g) + 0.5
    weight[torch.randperm(N, device="cuda", generator=g)[:case["masked"]]] = 0.0  # tokens without a loss
    s["weight"] = weight
    s["upstream"] = torch.rand(N, device="cuda", generator=g) + 0.5
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, g)
    if case["op"] == "top":
        return _prepare_top(case, g)
    return _prepare_distill(case, g)


# ---- the plain forms ----------------------------------------------------------------------------------

def _plain_sample(s):
    x = s["logits"].float()
    B, V = x.shape
    if "penalty" in s:
        seen = torch.zeros(B, V, dtype=torch.bool, device=x.device)
        rows = torch.arange(B, device=x.device).repeat_interleave(s["case"]["seen"])
        seen[rows, s["seen_ids"].long()] = True
        pen = s["penalty"][:, None]
        x = torch.where(seen, torch.where(x > 0, x / pen, x * pen), x)
    y = x / s["temperature"][:, None]
    y, order = torch.sort(y, dim=1, descending=True, stable=True)  # ties: the lower index first
    k = s["top_k"].long()[:, None]
    rank = torch.arange(V, device=x.device)[None, :]
    on = (k >= 1) & (k <= min(V, 1024))
    z = y.double() - y[:, :1].double()
    w = torch.exp(z) * (~on | (rank < k))
    cum = torch.cumsum(w, dim=1)
    p = s["top_p"].double()[:, None]
    keep = (w > 0) & ((cum - w < p * cum[:, -1:]) | (p >= 1))
    keep &= z >= torch.log(s["min_p"].double())[:, None]
    keep[:, 0] = True
    score = torch.where(keep, w / (s["q"].gather(1, order).double() + 1e-20), torch.full_like(w, -1.0))
    best = score.amax(dim=1, keepdim=True)
    return torch.where(score == best, order, V).amin(dim=1)  # the lower index of equal scores


def _plain_logsumexp(a):
    m = a.amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    return torch.log(torch.exp(a - m).sum(dim=1, dtype=torch.float64)) + m[:, 0].double()


def _plain_top(s):
    n, tau = s["case"]["n"], s["case"]["tau"]
    x = s["logits"].float()
    values, order = torch.sort(x, dim=1, descending=True, stable=True)  # ties: the lower index first
    a = values / tau
    lse = _plain_logsumexp(a)
    rest = _plain_logsumexp(a[:, n:]) if n < x.shape[1] else torch.full_like(lse, -math.inf)
    logprob = x.gather(1, s["tokens"][:, None])[:, 0] / tau - lse
    return dict(ids=order[:, :n].to(torch.int32), values=values[:, :n].clone(), lse=lse.float(), rest=rest.float(), logprob=logprob.float())


def _plain_distill(s, scale, grad):
    """The loss of every row times its weight, and with grad the gradient for upstream gradients `scale`."""
    tau, r = s["case"]["tau"], s["rest"]
    a = s["student"].float()
    m = a.amax(dim=1, keepdim=True)
    a = (a - m) / tau  # L and R are relative to the row's maximum
    N, V = a.shape
    valid = (s["ids"] >= 0) & (s["ids"] < V)
    ids = torch.where(valid, s["ids"], 0).long()
    t = torch.where(valid, s["values"].double() / tau, -math.inf)
    if r is not None:
        t = torch.cat([t, r.double()[:, None]], dim=1)
    counts = valid.any(dim=1) & (s["weight"] != 0)
    t = torch.where(counts[:, None], t, 0.0)
    e = torch.exp(t - t.amax(dim=1, keepdim=True))
    p = e / e.sum(dim=1, keepdim=True)
    L = _plain_logsumexp(a)
    member = torch.zeros(N, V + 1, dtype=torch.bool, device=a.device)
    member.scatter_(1, torch.where(valid, ids, V), True)
    member = member[:, :V]
    logq = (s["student"].gather(1, ids).double() - m.double()) / tau - L[:, None]
    if r is not None:
        R = _plain_logsumexp(a.masked_fill(member, -math.inf))
        logq = torch.cat([logq, (R - L)[:, None]], dim=1)
    term = torch.where(p > 0, p * (torch.log(p) - logq), 0.0).sum(dim=1)
    loss = torch.where(counts, s["weight"] * tau * tau * term, 0.0).float()
    if not grad:
        return loss
    d = torch.exp(a - L[:, None].float())
    if r is not None:
        d -= torch.where(member, 0.0, torch.exp(a - R[:, None].float()) * p[:, -1:].float())
    d.scatter_add_(1, ids, torch.where(valid, -p[:, :ids.shape[1]].float(), 0.0))
    d *= torch.where(counts, scale * s["weight"] * tau, 0.0)[:, None]
    return dict(loss=loss, grad=d.to(s["student"].dtype))


def _plain(s):
    op = s["case"]["op"]
    if op == "sample":
        return _plain_sample(s)
    if op == "top":
        return _plain_top(s)
    if op == "loss":
        return _plain_distill(s, None, False)
    return _plain_distill(s, s["upstream"] if op == "autograd" else torch.ones_like(s["weight"]), True)


# ---- the framework's calls ----------------------------------------------------------------------------

def _own(s):
    import decode_token_sampling_gb300 as kps

    case = s["case"]
    if case["op"] == "sample":
        idx, _ = kps.sample(s["logits"], s["top_k"], s["top_p"], s["temperature"], s["q"], min_p=s["min_p"],
                            seen_indptr=s.get("seen_indptr"), seen_ids=s.get("seen_ids"), penalty=s.get("penalty"),
                            workspace=s["workspace"])
        return idx
    if case["op"] == "top":
        t = kps.top_logits(s["logits"], case["n"], temperature=case["tau"], tokens=s["tokens"])
        return dict(ids=t.ids, values=t.values, lse=t.lse, rest=t.rest, logprob=t.logprob)
    kw = dict(temperature=case["tau"], rest=s["rest"], weight=s["weight"])
    if case["op"] == "loss":
        return kps.distill_loss(s["student"], s["ids"], s["values"], **kw)
    if case["op"] == "step":
        loss, grad = kps.distill_loss_grad(s["student"], s["ids"], s["values"], **kw)
        return dict(loss=loss, grad=grad)
    student = s["student"].detach().requires_grad_()
    loss = kps.distill_loss(student, s["ids"], s["values"], **kw)
    grad, = torch.autograd.grad(loss, student, s["upstream"])
    return dict(loss=loss.detach(), grad=grad)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        n = case["B"] * case["V"]
        return dict(bytes=n * b + case["B"] * (28 + 4 * case["seen"]), flops=4 * n)
    if case["op"] == "top":
        n = case["B"] * case["V"]
        return dict(bytes=n * b + case["B"] * (8 * case["n"] + 20), flops=4 * n)
    rows = case["N"] - case["masked"]
    small = case["N"] * (8 + 4 * bool(case["rest"])) + rows * case["K"] * (4 + b)
    if case["op"] == "loss":
        return dict(bytes=rows * case["V"] * b + small, flops=4 * rows * case["V"])
    return dict(bytes=(rows + case["N"]) * case["V"] * b + small, flops=8 * rows * case["V"])


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def _exact_top(s):
    x, n, tau = s["logits"], s["case"]["n"], s["case"]["tau"]
    out = dict(ids=None, values=[], lse=[], rest=[], logprob=[])
    for at in range(0, x.shape[0], 64):
        d = x[at:at + 64].double()
        a = d / tau
        lse = torch.logsumexp(a, 1)
        top = torch.topk(d, n, dim=1)
        out["values"].append(top.values)
        out["lse"].append(lse)
        out["rest"].append(torch.logsumexp(a.scatter(1, top.indices, -math.inf), 1))
        out["logprob"].append(a.gather(1, s["tokens"][at:at + 64, None])[:, 0] - lse)
    return {k: None if v is None else torch.cat(v) for k, v in out.items()}


def _exact_distill(s):
    op, tau = s["case"]["op"], s["case"]["tau"]
    losses, grads = [], []
    for at in range(0, s["student"].shape[0], 128):
        rows = slice(at, at + 128)
        a = s["student"][rows].double() / tau
        n, V = a.shape
        w = s["weight"][rows].double()
        ids, val = s["ids"][rows].long(), s["values"][rows].double() / tau
        # teacher's masses by token (column V: empty slots), then the rest's
        ok = (ids >= 0) & (ids < V)
        where = torch.where(ok, ids, V)
        log_t = torch.where(ok, val, -math.inf)
        r = s["rest"][rows].double()[:, None] if s["rest"] is not None else torch.full((n, 1), -math.inf, device=a.device, dtype=a.dtype)
        live = (ok.any(1) & (w != 0)).double()
        Z = torch.logsumexp(torch.cat([log_t, r, torch.where(live == 0, 0.0, -math.inf)[:, None]], 1), 1, keepdim=True)
        logp = torch.log_softmax(a, 1)
        token_p = torch.zeros(n, V + 1, device=a.device, dtype=a.dtype).scatter_add_(1, where, torch.exp(log_t - Z))[:, :V]
        in_list = torch.zeros(n, V + 1, device=a.device, dtype=torch.bool).scatter_(1, where, True)[:, :V]
        log_rest = torch.logsumexp(logp.masked_fill(in_list, -math.inf), 1, keepdim=True)
        pt, pr = torch.exp(log_t - Z), torch.exp(r - Z)
        picked = torch.gather(logp, 1, torch.where(ok, ids, 0))
        kl = torch.where(pt > 0, pt * (log_t - Z - picked), 0.0).sum(1) + torch.where(pr > 0, pr * (r - Z - log_rest), 0.0)[:, 0]
        losses.append(torch.where(live > 0, w * tau ** 2 * kl, 0.0))
        if op != "loss":
            share = torch.exp(logp - log_rest).masked_fill(in_list, 0.0)  # of the student's rest
            up = s["upstream"][rows].double() if op == "autograd" else 1.0
            grads.append((torch.exp(logp) - token_p - pr * share) * (live * w * tau * up)[:, None])
    loss = torch.cat(losses)
    return loss if op == "loss" else dict(loss=loss, grad=torch.cat(grads))


def exact(case, seed):
    if case["op"] == "sample":
        return None  # token ids
    s = prepare(case, seed)
    return _exact_top(s) if case["op"] == "top" else _exact_distill(s)
