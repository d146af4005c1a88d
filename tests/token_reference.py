"""Plain 64-bit forms of the operators on given tokens, and how far the kernels may be from them.

With d_v = (x_v - max) / T, eps = sum of exp(d_v) over all but one largest element and Q = -sum p_v d_v,
the bounds count the kernels' roundings (u = 2^-24, half a step of fp32, relative):
  * an exponent (x - m) c: the difference, the product and the two roundings of c, 4 u |d| on the
    exponential, which itself is right to 2^-22 (ex2.approx);
  * a sum of them by 256 threads: two additions to an accumulator a vector of G elements, 2 V / (256 G),
    up to 160 of listed elements and of merges;
  * a reference that rises: once in each of a thread's rounds of six vectors at most, and in the
    merges, each an exponential and two products.
"""

import math

import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22
TINY = 1e-30  # what lies 2^-126 below a row's largest is taken as zero, at most 2^20 times


def _relative(V, bf16):
    G = 8 if bf16 else 4
    rounds = math.ceil(V / (256 * 6 * G))
    return EX2 + (2 * V / (256 * G) + 160) * U + (rounds + 6) * (EX2 + 2 * U)


def temperatures(temperature, N, device):
    """Per row, as the operators take them: what is no positive normal number counts as 1."""
    t = temperature if isinstance(temperature, torch.Tensor) else torch.full((N,), temperature, dtype=torch.float64, device=device)
    t = t.double()
    if isinstance(temperature, torch.Tensor):
        t = torch.where((t >= torch.finfo(torch.float32).tiny) & (t < math.inf), t, 1.0)
    return t[:, None]


class Rows:
    """The quantities of every row in float64, with their bounds."""

    def __init__(self, logits, tokens, temperature=1.0):
        x = logits.double()
        N, V = x.shape
        self.T = T = temperatures(temperature, N, x.device)
        self.live = (tokens >= 0) & (tokens < V)
        self.at = torch.where(self.live, tokens, 0)[:, None]
        top = torch.where(torch.isnan(x), -math.inf, x).amax(1, keepdim=True)
        self.ok = torch.isfinite(top[:, 0]) & ~torch.isnan(x).any(1) & ~(x == math.inf).any(1)
        m = torch.where(self.ok[:, None], top, 0.0)
        x = torch.where(self.ok[:, None], x, 0.0)  # rows without a distribution are overwritten at the end
        self.d = d = (x - m) / T
        first = (x == m).to(torch.uint8).argmax(1, keepdim=True)
        e = torch.exp(d)
        others = e.scatter(1, first, 0.0)
        self.eps = eps = others.sum(1)
        weighted = torch.where(e > 0, e * -d, 0.0)
        self.S = S = 1 + eps
        self.Q = Q = weighted.sum(1) / S
        self.lse = torch.log1p(eps)
        self.entropy = self.lse + Q
        self.p = e / S[:, None]
        # bounds
        rel = _relative(V, logits.dtype == torch.bfloat16)
        squares = torch.where(e > 0, e * d * d, 0.0).sum(1)
        self.r1 = rel + 4 * U * weighted.sum(1) / eps.clamp(min=1e-300)
        self.r2 = rel + 4 * U + 4 * U * squares / weighted.sum(1).clamp(min=1e-300)
        self.share = self.r1 * eps / S  # of S
        self.lse_tol = self.share + 4 * U * self.lse
        self.entropy_tol = self.lse_tol + Q * (self.r1 + self.r2 + 4 * U) + U * self.entropy + TINY
        self.at_max = d.gather(1, self.at)[:, 0] == 0

    def logprob(self, index):
        """Log-probabilities at index [N, k], and their bounds."""
        d = self.d.gather(1, index)
        lp = d - self.lse[:, None]
        tol = 2 * U * d.abs().nan_to_num(posinf=0.0) + self.lse_tol[:, None] + U * lp.abs().nan_to_num(posinf=0.0) + TINY
        return torch.where(self.ok[:, None], lp, math.nan), tol

    def grad(self, g, h, g_tol=None, h_tol=None):
        """The gradient for those of the log-probability and the entropy [N], and its bound before its own
        rounding."""
        zero = torch.zeros_like(self.eps)
        g, h = (zero if t is None else t.double() for t in (g, h))
        p, d, T, Q = self.p, self.d, self.T, self.Q[:, None]
        delta = torch.zeros_like(p).scatter_(1, self.at, 1.0)
        one_less = torch.where(delta > 0, torch.where(self.at_max, self.eps / self.S, 1 - p.gather(1, self.at)[:, 0])[:, None], -p)
        info = torch.where(p > 0, p * (d + Q), 0.0)
        grad = (g[:, None] * one_less - h[:, None] * info) / T
        size = torch.where(p > 0, d.abs(), 0.0)
        rel = EX2 + 4 * U * size + self.share[:, None] + 8 * U
        ga, ha = g.abs()[:, None], h.abs()[:, None]
        # (Q's terms below 2^-126 are zero too: at most 2^20 of 2^-126 times an exponent of 88, 1.1e-30)
        tol = p * (ga + ha * (size + Q)) * rel + p * ha * (Q * (self.r1 + self.r2)[:, None] + 2 * TINY) + 4 * U * p * ha * size
        # the token's own: eps / S where it is the largest (its terms below 2^-126 are zero: at most 2^20 of them,
        # 1.3e-32), else 1 - p of a p of at most 1/2
        own = torch.where(self.at_max, (self.eps / self.S) * (self.r1 + 6 * U) + TINY, 2 * U + p.gather(1, self.at)[:, 0] * rel.gather(1, self.at)[:, 0])
        tol = tol + delta * ga * own[:, None] + 4 * U * (ga * one_less.abs() + ha * info.abs())
        if g_tol is not None:
            tol = tol + g_tol[:, None] * one_less.abs()
        if h_tol is not None:
            tol = tol + h_tol[:, None] * info.abs()
        tol = (tol + (ga + 200 * ha) * 1e-37) / T + 1e-44
        on = self.live & ((g != 0) | (h != 0))
        grad = torch.where(on[:, None], torch.where(self.ok[:, None], grad, math.nan), 0.0)
        return grad, torch.where(on[:, None], tol, 0.0)


def score_reference(logits, tokens, n=0, temperature=1.0):
    """dict of logprob, entropy, rank, ids, logprobs with bounds under name + "_tol"."""
    r = Rows(logits, tokens, temperature)
    lp, lp_tol = r.logprob(r.at)
    live, dead = r.live, ~r.live
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    out = dict(logprob=lp[:, 0].masked_fill(dead, 0.0), logprob_tol=lp_tol[:, 0],
               entropy=torch.where(r.ok, r.entropy, math.nan).masked_fill(dead, 0.0), entropy_tol=r.entropy_tol,
               rank=(x > x.gather(1, r.at)).sum(1).to(torch.int32).masked_fill(dead, -1))
    if n:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :n]
        top, tol = r.logprob(order)
        out.update(ids=order.to(torch.int32).masked_fill(dead[:, None], -1),
                   logprobs=top.masked_fill(dead[:, None], -math.inf), logprobs_tol=tol)
    return out


def policy_reference(logits, tokens, old, advantage, clip=(0.2, 0.2), ref=None, kl=0.0, ent=0.0, weight=None, temperature=1.0):
    """dict of loss, logprob, entropy, grad with bounds under name + "_tol"."""
    r = Rows(logits, tokens, temperature)
    w = torch.ones_like(r.eps) if weight is None else weight.double()
    r.live = r.live & (w != 0)
    lp, lp_tol = (t[:, 0] for t in r.logprob(r.at))
    old, A = old.double(), advantage.double()
    lo, hi = (torch.tensor(v, dtype=torch.float32) for v in clip)  # the bounds are fp32 sums
    lo, hi = float(1 - lo), float(1 + hi)
    ratio = torch.exp(lp - old)
    ratio_tol = ratio * (lp_tol + U * (lp - old).abs().nan_to_num(posinf=0.0) + 4 * U)
    clipped = torch.where(A >= 0, ratio > hi, ratio < lo)
    v = torch.where(A == 0, 0.0, -torch.minimum(ratio * A, ratio.clamp(lo, hi) * A))
    g = torch.where(clipped | (A == 0), 0.0, -A * ratio)
    g_tol = torch.where(clipped | (A == 0), 0.0, A.abs() * ratio_tol) + U * g.abs()
    v_tol = g_tol + 2 * U * v.abs()
    size = v.abs()
    if kl:
        kl = float(torch.tensor(kl, dtype=torch.float32))
        u = ref.double() - lp
        u_tol = lp_tol + U * u.abs()
        e = torch.expm1(u)
        k3 = e - u
        v, g = v + kl * k3, g - kl * e
        v_tol = v_tol + abs(kl) * (e.abs() * u_tol + u_tol ** 2 + 12 * U * k3 + torch.where(u.abs() < 0.5, 0.0, U * (5 * e.abs() + u.abs())))
        g_tol = g_tol + abs(kl) * ((1 + e) * u_tol + 5 * U * e.abs())
        size = size + abs(kl) * k3
    h = h_tol = torch.zeros_like(w)
    if ent:
        ent = float(torch.tensor(ent, dtype=torch.float32))
        v = v - ent * r.entropy
        v_tol = v_tol + abs(ent) * r.entropy_tol
        size = size + abs(ent) * r.entropy
        h = -w * ent
        h_tol = U * h.abs()
    g, g_tol = w * g, w.abs() * (g_tol + 2 * U * g.abs())
    grad, grad_tol = r.grad(g, h, g_tol, h_tol)
    zero = (r.live & ~r.ok)[:, None]
    grad = torch.where(zero, math.nan, grad)
    live = r.live
    pick = lambda t, tol: (torch.where(live, torch.where(r.ok, t, math.nan), 0.0), torch.where(live, tol, 0.0))  # noqa: E731
    out = {}
    out["loss"], out["loss_tol"] = pick(w * v, w.abs() * (v_tol + 5 * U * size) + TINY)
    out["logprob"], out["logprob_tol"] = pick(lp, lp_tol)
    out["entropy"], out["entropy_tol"] = pick(r.entropy, r.entropy_tol)
    # a gradient whose factors are both 0 is 0 where the row is a distribution
    out["grad"], out["grad_tol"] = grad, torch.where(live[:, None], grad_tol, 0.0)
    return out


def close(got, want, tol, what):
    """NaN and infinities alike, everything else within tol.  What lies beyond the type's largest value
    rounds to infinity."""
    want = torch.where(want.abs() > torch.finfo(got.dtype).max, want * math.inf, want)
    got = got.double()
    special = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(same[special].all()), f"{what}: NaN or infinities differ"
    off = (got - want).abs()
    bad = ~special & ~(off <= tol)
    if bool(bad.any()):
        i = int(torch.where(bad, off / (tol + 1e-300), 0.0).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bounds, the worst at {i}: got "
                             f"{float(got.flatten()[i]):.9g}, want {float(want.flatten()[i]):.9g}, bound {float(tol.flatten()[i]):.3g}")


def close_grad(got, want, tol, what="grad"):
    """A gradient rounded once to its type."""
    half = torch.finfo(got.dtype).eps / 2
    small = torch.finfo(got.dtype).smallest_normal * half  # half a step below the normal numbers
    size = want.abs().nan_to_num(posinf=0.0)
    close(got, want, tol * (1 + half) + half * size + small, what)
