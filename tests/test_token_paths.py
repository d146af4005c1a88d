"""The ways through the kernels on given tokens that only some sizes and buffers take: the policy loss of rows too long for a
cluster's shared memory (two launches, the statistics in the outputs between them), and gradients whose rows do not share the
logits' 16-byte boundaries."""

import ctypes
import math

import pytest
import torch

from test_policy_loss import _case, check, own
from test_token_logprobs import _hard_rows, make, upstream
from token_reference import Rows, close, close_grad

gpu = pytest.mark.gpu
LONG = [(torch.float32, 500001), (torch.bfloat16, 917600), (torch.float32, 1 << 20)]  # eight CTAs hold 458752 and 917504
p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@gpu
@pytest.mark.parametrize("dtype,V", LONG[:2])
def test_hard_rows_in_two_launches(dtype, V):
    x, at = _hard_rows(dtype, V, 3)
    s = _case(20, V, dtype, seed=1)
    s["logits"] = x
    finite = torch.where(torch.isnan(x) | (x == math.inf), -math.inf, x)
    top = finite.argmax(1)
    for tokens in (top, at[:20]):
        r = Rows(x, tokens)
        lp, tol = (t[:, 0] for t in r.logprob(r.at))
        base = torch.where(torch.isfinite(lp), lp, -1.0).float()
        # A log-probability of -1e30 (the row of logits times 1e30, with a token that is not its largest) has a step of 2^76 in
        # fp32: that of the old policy is off by up to half of it, so that the ratio, the exponential of the difference, may be
        # anything from 0 to infinity and the loss either side of its clip.  policy_reference's bound, the ratio times that
        # of the log-probability, is one while the latter is small (exp(0.01) - 1 is 0.01 to half a per cent).  Beyond, only the
        # log-probability and the entropy are compared.
        sure = ~(tol > 0.01) | ~torch.isfinite(lp)
        assert int((~sure).sum()) == (0 if tokens is top else 1) and bool((lp[~sure] < -1e28).all())
        for old, ref, weight, kl, ent in ((base + 0.03, base + 0.3, s["weight"], 0.1 if tokens is top else 0.0, 0.05),
                                          (base - 0.5, base, None, 0.0, -0.2)):
            t = dict(s, tokens=tokens, old=old, ref=ref, weight=weight)
            got = own(t, kl=kl, ent=ent)
            close(got.logprob, lp, tol, "logprob")
            close(got.entropy, torch.where(r.ok, r.entropy, math.nan), r.entropy_tol, "entropy")
            check({k: v if v is None else v[sure] for k, v in t.items()}, kl=kl, ent=ent, got=type(got)(*(v[sure] for v in got)))


@gpu
@pytest.mark.parametrize("dtype,V", LONG)
def test_two_launches_repeat_in_graphs_and_on_streams(dtype, V):
    s = _case(3, V, dtype, seed=4, empty=1)
    want = check(s)
    side = torch.cuda.Stream()
    runs = [own(s, stream=side), own(s), own(s, stream=side)]
    torch.cuda.synchronize()
    graphs, live = [], {k: torch.zeros_like(v) for k, v in s.items()}
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            runs.append(own(live))
        graphs.append(graph)
    for k, v in s.items():
        live[k].copy_(v)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("dtype,V", LONG[:2])
def test_two_launches_with_a_gradient_of_another_phase(dtype, V):
    import decode_token_sampling_gb300 as kps
    N, ld = 3, V + 5
    s = _case(N, V, dtype, seed=5, empty=1)
    out = torch.full((3, N + 2), -5.0, device="cuda")
    buf = torch.full((N * ld + 9,), -5.0, dtype=dtype, device="cuda")
    st = kps.load_library().kps_policy_loss_grad(
        p(s["logits"]), 0 if dtype == torch.float32 else 1, N, V, V, p(s["tokens"]), 1.0, None, p(s["old"]), p(s["advantage"]), p(s["ref"]),
        p(s["weight"]), 0.2, 0.28, 0.1, 0.05, p(out[0]), p(out[1]), p(out[2]), p(buf[3:]), ld, _stream())
    assert st == 0
    rows = buf[3:3 + N * ld].view(N, ld)
    check(s, got=kps.PolicyLoss(out[0, :N], rows[:, :V], out[1, :N], out[2, :N]))
    assert bool((out[:, N:] == -5).all())
    assert bool((buf[:3] == -5).all()) and bool((buf[3 + N * ld:] == -5).all()) and bool((rows[:, V:] == -5).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,ld", [(5, 5003, 5010), (1, 3, 3), (2, 100001, 100003), (200, 1001, 1001), (2, 1 << 20, (1 << 20) + 1)])
def test_gradients_of_logprobs_of_another_phase(N, V, ld, dtype):
    """Rows of one block and rows split over a cluster; nothing is written between or behind the rows."""
    import decode_token_sampling_gb300 as kps
    x, tokens = make(N, V, dtype, seed=V)
    if N > 2:
        tokens[1], tokens[2] = -1, V - 1
    g, h = upstream(N)
    _, stats = kps.token_logprobs_forward(x, tokens, temperature=0.8)
    for shift in (1, 3):
        for gg, hh in ((g, h), (g, None), (None, h)):
            buf = torch.full((N * ld + 9,), -5.0, dtype=dtype, device="cuda")
            st = kps.load_library().kps_token_logprobs_backward(
                p(x), 0 if dtype == torch.float32 else 1, N, V, V, p(tokens), 0.8, None, None if gg is None else p(gg),
                None if hh is None else p(hh), p(stats), p(buf[shift:]), ld, _stream())
            assert st == 0
            rows = buf[shift:shift + N * ld].view(N, ld)
            want, tol = Rows(x, tokens, float(torch.tensor(0.8))).grad(gg, hh)
            close_grad(rows[:, :V], want, tol)
            assert bool((buf[:shift] == -5).all()) and bool((buf[shift + N * ld:] == -5).all()) and bool((rows[:, V:] == -5).all())
