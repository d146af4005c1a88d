"""Plain 64-bit forms of the operators on rows of logits, and how far the kernels may be from them.

The bounds count the kernels' roundings (u = 2^-24, half a step of fp32, relative):
  * an exponent z = (x - ref) c: the difference, the product and c itself, 3 u |z|;
  * an exponential: 2^-22 relative (ex2.approx), times what its exponent's error makes of it;
  * a sum of n of them by 256 threads: each thread adds n / (256 G) vectors of G elements in
    turn, at most 4 + 1 additions deep inside a vector, and 8 + 3 merges follow, each merge two
    exponentials deep: (n / (256 G) + 16) u + 11 * 2^-21 for rows that merge unequal references.
"""

import math

import torch

U = 2.0 ** -24
EX2 = 2.0 ** -22


def sum_error(V, bf16=True):
    G = 8 if bf16 else 4
    return EX2 + (V / (256 * G) + 16) * U + 11 * 2 * EX2


def distill_reference(student, ids, values, tau, rest=None, weight=None, upstream=None):
    """(loss, grad, loss_tol, grad_tol) in float64: the formulas, and the largest errors the fp32
    kernel may make before the gradient's own rounding."""
    s = student.double()
    N, V = s.shape
    dev = s.device
    a = s / tau
    t = values.double() / tau
    ok = (ids >= 0) & (ids < V) & ~(values == -math.inf)
    w = torch.ones(N, dtype=torch.float64, device=dev) if weight is None else weight.double()
    live = ok.any(1) & (w != 0)
    t = torch.where(ok, t, -math.inf)
    r = torch.full((N, 1), -math.inf, dtype=torch.float64, device=dev) if rest is None else rest.double()[:, None]
    classes = torch.cat([t, r], 1)
    classes = torch.where(live[:, None], classes, 0.0)
    p = torch.softmax(classes, 1)
    logp = torch.log_softmax(classes, 1)
    col = torch.where(ok, ids.long(), V)
    member = torch.zeros(N, V + 1, dtype=torch.bool, device=dev).scatter_(1, col, True)[:, :V]
    pv = torch.zeros(N, V + 1, dtype=torch.float64, device=dev).scatter_add_(1, col, torch.where(ok, p[:, :-1], 0.0))[:, :V]
    L = torch.logsumexp(a, 1, keepdim=True)
    outside = a.masked_fill(member, -math.inf)
    R = torch.logsumexp(outside, 1, keepdim=True)
    logq = torch.cat([a.gather(1, torch.where(ok, ids.long(), 0)) - L, R - L], 1)
    terms = torch.where(p > 0, p * (logp - logq), 0.0)
    kl = terms.sum(1)
    # a student's row that has no distribution
    bad = ~torch.isfinite(L[:, 0]) | torch.isnan(s).any(1)
    kl = torch.where(bad, math.nan, kl)
    loss = torch.where(live, w * tau * tau * kl, 0.0)
    q = torch.exp(a - L)
    share = torch.where(member, 0.0, torch.exp(outside - R)) if rest is not None else torch.zeros_like(q)
    share = torch.where(p[:, -1:] > 0, share, 0.0)
    scale = w * tau
    up = None if upstream is None else upstream.double()
    if up is not None:
        scale = scale * up
        live = live & (scale != 0)
    g = q - pv - p[:, -1:] * share
    g = torch.where(bad[:, None], math.nan, g)
    grad = torch.where(live[:, None], scale[:, None] * g, 0.0)
    # bounds: D is the reach of the exponents that carry mass
    d = sum_error(V, student.dtype == torch.bfloat16)
    ref = torch.where(ok, a.gather(1, torch.where(ok, ids.long(), 0)), -math.inf).amax(1, keepdim=True)
    tref = classes.amax(1, keepdim=True)
    reach_k = torch.where(p > 0, (classes - tref).abs() + (logq + L - ref).abs(), 0.0)
    D = (torch.nan_to_num(reach_k, posinf=0.0) * p).sum(1) + torch.nan_to_num((L - ref).abs()[:, 0], posinf=0.0)
    Z = (p * (1 + 3 * torch.nan_to_num((classes - tref).abs(), posinf=0.0) * U / EX2)).sum(1) * EX2  # error of the p's
    span = torch.nan_to_num((logp - logq).abs(), posinf=0.0, nan=0.0)
    worst = torch.where(p > 1e-30, span, 0.0).amax(1)
    loss_tol = (w * tau * tau).abs() * (16 * U * (D + 1) + 3 * d + 4 * (Z + 24 * U) * (worst + 1)) + 4 * U * loss.abs()
    mv = torch.nan_to_num((a - a.amax(1, keepdim=True)).abs(), posinf=0.0, nan=0.0).clamp(max=200.0)
    rel = 2 * d + EX2 * 4 + 6 * U * (mv + 1) + 6 * U * torch.nan_to_num((L - ref).abs(), posinf=0.0, nan=0.0)
    prel = (4 * EX2 + 8 * U * (classes - tref).abs().nan_to_num(posinf=0.0).clamp(max=200.0).amax(1, keepdim=True)) + 2 * d
    grad_tol = scale.abs()[:, None] * ((q + p[:, -1:] * share) * rel + (pv + p[:, -1:] * share) * prel) + 1e-37
    # rows without a loss are zero to the bit, whatever the student holds there
    loss_tol = torch.where(live, loss_tol, 0.0)
    grad_tol = torch.where(live[:, None], grad_tol, 0.0)
    return loss, grad, loss_tol, grad_tol


def top_reference(logits, n, tau, tokens=None):
    """ids, values, lse, rest, logprob in float64 (NaN as -inf)."""
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    values, order = torch.sort(x, dim=1, descending=True, stable=True)
    a = values / tau
    lse = torch.logsumexp(a, 1)
    rest = torch.logsumexp(a[:, n:], 1) if n < x.shape[1] else torch.full_like(lse, -math.inf)
    out = dict(ids=order[:, :n].to(torch.int32), values=values[:, :n], lse=lse, rest=rest)
    if tokens is not None:
        V = x.shape[1]
        inside = (tokens >= 0) & (tokens < V)
        got = x.gather(1, torch.where(inside, tokens, 0)[:, None])[:, 0] / tau - lse
        out["logprob"] = torch.where(inside, got, -math.inf)
    return out
