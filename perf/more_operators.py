"""Cases for the operators on the tokens of a policy beside the sampling step: the log-probabilities of given tokens
with their ranks, the entropy and the top alternatives of their rows; the gradient of those; and the clipped policy
loss with its gradient.

Where `own` is false, `run` computes them in plain torch operations; where it is true it calls
decode_token_sampling_gb300.
"""

import math

import torch

own = False

BIG_V = 151936


def listed():
    return [
        # log-probabilities: one sequence decoding; a serving batch at temperatures of its own, 20 alternatives each; a
        # prompt scored with five; a long list over odd rows in a padded buffer; an old policy's pass over a batch of
        # rollouts, a quarter of whose rows are padding
        _logprobs("logprobs one row", 1, BIG_V, 5, "f32"),
        _logprobs("logprobs serving batch", 256, BIG_V, 20, "bf16", temps=True),
        _logprobs("logprobs prompt", 2048, 128256, 5, "bf16"),
        _logprobs("logprobs long list odd", 96, 50001, 1000, "f32", ld=50048, tau=0.7, pad=49),
        _logprobs("logprobs rollouts", 4096, BIG_V, 0, "bf16", empty=1024),
        # the same with the gradient of log-probabilities and entropies through autograd: a small batch, odd rows, a
        # training batch
        _train("autograd", "autograd small", 64, 32000, "f32"),
        _train("autograd", "autograd odd", 333, 50001, "f32", tau=0.7, empty=60),
        _train("autograd", "autograd batch", 2048, 128256, "bf16", empty=512),
        # the policy loss with its gradient: a small batch, odd rows in a padded buffer, a training batch with every
        # term, one of the clipped term alone
        _train("policy", "policy small", 16, 32000, "f32", kl=0.05),
        _train("policy", "policy odd", 130, 50001, "f32", ld=50048, tau=0.9, empty=30, kl=0.05, ent=0.01),
        _train("policy", "policy batch", 4096, BIG_V, "bf16", empty=1024, kl=0.02, ent=0.003),
        _train("policy", "policy batch clipped term", 2048, 128256, "bf16"),
    ]


def _logprobs(name, N, V, n, dtype, ld=None, tau=1.0, temps=False, pad=0, empty=0):
    return dict(name=name, op="logprobs", N=N, V=V, ld=ld or V, n=n, dtype=dtype, tau=tau, temps=temps, pad=pad, empty=empty)


def _train(op, name, N, V, dtype, ld=None, tau=1.0, temps=False, pad=0, empty=0, kl=0.0, ent=0.0):
    return dict(name=name, op=op, N=N, V=V, ld=ld or V, dtype=dtype, tau=tau, temps=temps, pad=pad, empty=empty, kl=kl, ent=ent)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "autograd", "policy"])
    N, V = _log(rng, 1, 2048), _log(rng, 1000, BIG_V)
    dtype = rng.choice(["f32", "bf16"])
    kw = dict(ld=rng.choice([V, -(-V // 64) * 64]), tau=rng.choice([0.7, 1.0, 1.3]), temps=rng.random() < 0.3,
              pad=rng.choice([0, rng.randint(1, 200)]), empty=rng.choice([0, N // 4]))
    if op == "logprobs":
        n = rng.choice([0, _log(rng, 1, 30), _log(rng, 1, min(V, 1024))])
        case = _logprobs("", N, V, n, dtype, **kw)
    elif op == "autograd":
        case = _train(op, "", N, V, dtype, **kw)
    else:
        case = _train(op, "", N, V, dtype, **kw, kl=rng.choice([0.0, 0.03]), ent=rng.choice([0.0, 0.01]))
    del case["name"]
    return case


# ---- inputs ------------------------------------------------------------------------------------------

CLIP = (0.2, 0.28)


def prepare(case, seed):
    """Rows of logits from near certain to flat, with tokens sampled from them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    N, V, ld = case["N"], case["V"], case["ld"]
    # N(0, 2.5) plus a bonus of 4 to 16 a row over the root of a rank drawn per token; the columns behind V hold junk
    x = torch.randn(N, ld, device="cuda", generator=g).mul_(2.5)
    bonus = torch.rand(N, 1, device="cuda", generator=g).mul_(12.0).add_(4.0)
    x.addcmul_(torch.rand(N, ld, device="cuda", generator=g).mul_(V).add_(1.0).rsqrt_(), bonus)
    if case["pad"]:
        x[:, V - case["pad"]:V] = -math.inf  # columns that pad the vocabulary
    x = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)[:, :V]
    u = lambda lo, hi: torch.rand(N, device="cuda", generator=g) * (hi - lo) + lo  # noqa: E731
    s = dict(case=case, logits=x, temperature=u(0.5, 1.2) if case["temps"] else case["tau"])
    tau = s["temperature"][:, None] if case["temps"] else case["tau"]
    score = (x.float() / tau).sub_(torch.empty(N, V, device="cuda").exponential_(generator=g).log_())
    tokens = score.argmax(dim=1)
    del score
    clean = tokens.clone()
    tokens[torch.randperm(N, device="cuda", generator=g)[:case["empty"]]] = -100  # padding
    s["tokens"] = tokens
    normal = lambda sigma: torch.randn(N, device="cuda", generator=g) * sigma  # noqa: E731
    if case["op"] == "autograd":
        s["grad_logprob"], s["grad_entropy"] = normal(1.0), normal(0.1)
    if case["op"] == "policy":
        # the policy has moved since its tokens were sampled; no ratio within half a per cent of a clip's border
        lp = torch.empty(N, device="cuda")
        for at in range(0, N, 256):
            a = x[at:at + 256].float() / (tau[at:at + 256] if case["temps"] else tau)
            lp[at:at + 256] = a.gather(1, clean[at:at + 256, None])[:, 0] - a.logsumexp(1)
        step = normal(0.2)
        for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
            step = torch.where((step - border).abs() < 0.005, step + 0.01, step)
        s["old"] = lp - step
        s["advantage"] = normal(1.0)
        s["ref"] = lp + normal(0.1) if case["kl"] else None
        s["weight"] = u(0.5, 1.5)
    return s


# ---- the plain forms ----------------------------------------------------------------------------------

def _plain_rows(s):
    """Per row: log-probabilities [N, V], those of the tokens, entropies, and which rows have a token."""
    case = s["case"]
    tau = s["temperature"][:, None] if case["temps"] else case["tau"]
    x = s["logits"].float()
    live = (s["tokens"] >= 0) & (s["tokens"] < case["V"])
    at = torch.where(live, s["tokens"], 0)[:, None]
    a = x / tau
    a = a - a.amax(dim=1, keepdim=True)
    logp = a - torch.log(torch.exp(a).sum(dim=1, keepdim=True, dtype=torch.float64)).float()
    del a
    p = torch.exp(logp)
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(dim=1, dtype=torch.float64)
    return x, logp, p, logp.gather(1, at)[:, 0], entropy, live, at


def _plain_grad(s, p, logp, entropy, live, at, g, h):
    """The gradient of the logits for the tokens' gradients g and the entropies' h."""
    case = s["case"]
    tau = s["temperature"][:, None] if case["temps"] else case["tau"]
    d = p * -g[:, None]
    if h is not None:
        d -= torch.where(p > 0, p * (logp + entropy[:, None].float()), 0.0) * h[:, None]
    d.scatter_add_(1, at, g[:, None])
    return torch.where(live[:, None], d / tau, 0.0).to(s["logits"].dtype)


def _plain(s):
    case = s["case"]
    x, logp, p, lp, entropy, live, at = _plain_rows(s)
    out = dict(logprob=torch.where(live, lp, 0.0), entropy=torch.where(live, entropy, 0.0).float())
    if case["op"] == "logprobs":
        rank = (x > x.gather(1, at)).sum(dim=1)
        out["rank"] = torch.where(live, rank, -1).to(torch.int32)
        if case["n"]:
            order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["n"]]  # ties: the lower index first
            out["ids"] = torch.where(live[:, None], order, -1).to(torch.int32)
            out["logprobs"] = torch.where(live[:, None], logp.gather(1, order), -math.inf)
        return out
    if case["op"] == "autograd":
        out["grad"] = _plain_grad(s, p, logp, entropy, live, at, s["grad_logprob"], s["grad_entropy"])
        return out
    w, A = s["weight"], s["advantage"]
    ratio = torch.exp(lp - s["old"])
    clipped = torch.where(A >= 0, ratio > 1 + CLIP[1], ratio < 1 - CLIP[0])
    loss = -torch.minimum(ratio * A, ratio.clamp(1 - CLIP[0], 1 + CLIP[1]) * A)
    g = torch.where(clipped, 0.0, -A * ratio)
    if case["kl"]:
        u = (s["ref"] - lp).double()
        loss = loss + case["kl"] * (torch.exp(u) - u - 1).float()
        g = g + case["kl"] * (1 - torch.exp(u)).float()
    if case["ent"]:
        loss = loss - case["ent"] * entropy.float()
    out["loss"] = torch.where(live, w * loss, 0.0)
    out["grad"] = _plain_grad(s, p, logp, entropy, live, at, w * g, -case["ent"] * w if case["ent"] else None)
    return out


# ---- the framework's calls ----------------------------------------------------------------------------

def _own(s):
    import decode_token_sampling_gb300 as kps

    case = s["case"]
    if case["op"] == "logprobs":
        t = kps.token_logprobs(s["logits"], s["tokens"], case["n"], temperature=s["temperature"])
        out = dict(logprob=t.logprob, entropy=t.entropy, rank=t.rank)
        if case["n"]:
            out.update(ids=t.ids, logprobs=t.logprobs)
        return out
    if case["op"] == "autograd":
        x = s["logits"].detach().requires_grad_()
        t = kps.token_logprobs(x, s["tokens"], temperature=s["temperature"])
        grad, = torch.autograd.grad([t.logprob, t.entropy], x, [s["grad_logprob"], s["grad_entropy"]])
        return dict(logprob=t.logprob.detach(), entropy=t.entropy.detach(), grad=grad)
    t = kps.policy_loss_grad(s["logits"], s["tokens"], s["old"], s["advantage"], clip=CLIP, ref_logprob=s["ref"],
                             kl_coef=case["kl"], entropy_coef=case["ent"], weight=s["weight"], temperature=s["temperature"])
    return dict(logprob=t.logprob, entropy=t.entropy, loss=t.loss, grad=t.grad)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    rows, N, V = case["N"] - case["empty"], case["N"], case["V"]
    small = N * (8 + 4 * case["temps"])
    if case["op"] == "logprobs":
        return dict(bytes=rows * V * b + small + N * (12 + 8 * case["n"]), flops=6 * rows * V)
    # the gradient is written whole, the empty rows' zeros too
    small += N * (16 if case["op"] == "autograd" else 24 + 4 * (case["kl"] > 0))
    return dict(bytes=(rows + N) * V * b + small, flops=10 * rows * V)


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    parts = []
    for lo in range(0, case["N"], 128):
        rows = slice(lo, lo + 128)
        token = s["tokens"][rows]
        n, V = len(token), case["V"]
        T = s["temperature"][rows].double()[:, None] if case["temps"] else case["tau"]
        has = token >= 0
        pick = token.clamp(min=0)[:, None]
        logq = torch.log_softmax(s["logits"][rows].double() / T, 1)
        q = logq.exp()
        lp = logq.gather(1, pick)
        H = torch.special.entr(q).sum(1, keepdim=True)
        out = dict(logprob=(lp * has[:, None])[:, 0], entropy=(H * has[:, None])[:, 0])
        if case["op"] == "logprobs":
            if case["n"]:
                best = torch.topk(logq, case["n"], dim=1).values
                out["logprobs"] = best.masked_fill(~has[:, None], -math.inf)
            parts.append(out)
            continue
        if case["op"] == "autograd":
            dlp, dH = s["grad_logprob"][rows].double()[:, None], s["grad_entropy"][rows].double()[:, None]
        else:
            w, A = s["weight"][rows].double()[:, None], s["advantage"][rows].double()[:, None]
            r = torch.exp(lp - s["old"][rows].double()[:, None])
            best = torch.where(A > 0, torch.clamp(r, max=1 + CLIP[1]), torch.clamp(r, min=1 - CLIP[0]))  # of the min
            L = -best * A
            dlp = torch.where(best == r, -r * A, 0.0)
            if case["kl"]:
                u = s["ref"][rows].double()[:, None] - lp
                L = L + case["kl"] * (torch.expm1(u) - u)
                dlp = dlp - case["kl"] * torch.expm1(u)
            L = (L - case["ent"] * H) * w
            dlp, dH = dlp * w, torch.full_like(w, -case["ent"]) * w
            out["loss"] = (L * has[:, None])[:, 0]
        onehot = torch.zeros(n, V, dtype=torch.float64, device=q.device).scatter_(1, pick, 1.0)
        info = torch.special.entr(q) - q * H  # d entropy / d a
        out["grad"] = (dlp * (onehot - q) + dH * info) / T * has[:, None]
        parts.append(out)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["op"] == "logprobs":
        out["rank"] = None
        if case["n"]:
            out["ids"] = None
    return out
