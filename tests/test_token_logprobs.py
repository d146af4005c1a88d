"""The log-probabilities of given tokens with ranks, entropies, alternatives and their gradient
(kps_token_logprobs, kps_token_logprobs_backward) against 64-bit forms."""

import ctypes
import math

import pytest
import torch

from token_reference import Rows, close, close_grad, score_reference

FAKE = ctypes.c_void_p(1 << 20)
OUT = ctypes.c_void_p(1 << 30)
odd = lambda by: ctypes.c_void_p((1 << 20) + by)  # noqa: E731


# ---- without a GPU: refusals, and the reference's own gradient against differences --------------

@pytest.fixture(scope="module")
def lib():
    from decode_token_sampling_gb300 import build
    build.build()
    import decode_token_sampling_gb300 as kps
    return kps.load_library()


def _forward(lib, **over):
    args = dict(logits=FAKE, dt=0, N=4, V=100, ld=100, tokens=FAKE, n=8, tau=1.0, taus=None, logprob=OUT, entropy=OUT,
                rank=OUT, ids=OUT, logprobs=OUT, stats=OUT, stream=None)
    assert not set(over) - set(args)
    args.update(over)
    return lib.kps_token_logprobs(*args.values())


def _backward(lib, **over):
    args = dict(logits=FAKE, dt=0, N=4, V=100, ld=100, tokens=FAKE, tau=1.0, taus=None, g=None, h=None, stats=FAKE, grad=OUT,
                ld_grad=100, stream=None)
    assert not set(over) - set(args)
    args.update(over)
    return lib.kps_token_logprobs_backward(*args.values())


@pytest.mark.parametrize("call", [_forward, _backward])
def test_shared_refusals(lib, call):
    for bad in (dict(dt=2), dict(N=-1), dict(V=0), dict(ld=99), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan),
                dict(tau=math.inf), dict(tau=1e-40), dict(logits=None), dict(tokens=None), dict(logits=odd(2)), dict(tokens=odd(4)),
                dict(taus=odd(2)), dict(dt=1, logits=odd(1))):
        assert call(lib, **bad) == 1, bad
    assert call(lib, V=(1 << 20) + 1, ld=1 << 21) == 2
    assert call(lib, N=1 << 40) == 2
    assert call(lib, N=0, logits=None, tokens=None) == 0
    if not torch.cuda.is_available():  # valid calls: they fail only for want of a GPU
        assert call(lib) == 4
        assert call(lib, tau=-1.0, taus=FAKE) == 4  # the number is not used then
        assert call(lib, N=1, ld=0) == 4


def test_own_refusals(lib):
    for bad in (dict(n=-1), dict(n=101), dict(n=1025, V=5000, ld=5000), dict(ids=None), dict(logprobs=None), dict(logprob=odd(2)),
                dict(entropy=odd(2)), dict(rank=odd(1)), dict(ids=odd(2)), dict(logprobs=odd(2)), dict(stats=odd(2))):
        assert _forward(lib, **bad) == 1, bad
    for bad in (dict(stats=None), dict(stats=odd(2)), dict(g=odd(2)), dict(h=odd(2)), dict(grad=None), dict(ld_grad=99),
                dict(grad=ctypes.c_void_p((1 << 30) + 2)), dict(grad=FAKE), dict(grad=ctypes.c_void_p((1 << 20) + 4 * 399)),
                dict(grad=ctypes.c_void_p((1 << 20) - 4 * 399))):
        assert _backward(lib, **bad) == 1, bad
    if not torch.cuda.is_available():
        assert _forward(lib, n=0, ids=None, logprobs=None, logprob=None, entropy=None, rank=None, stats=None) == 4
        assert _backward(lib, grad=ctypes.c_void_p((1 << 20) + 4 * 400)) == 4


def test_binding_refuses_cpu_tensors():
    import decode_token_sampling_gb300 as kps
    x, t = torch.zeros(2, 10), torch.zeros(2, dtype=torch.int64)
    for call in (kps.token_logprobs, kps.token_logprobs_forward):
        with pytest.raises(ValueError, match="CUDA"):
            call(x, t)
    with pytest.raises(ValueError, match="CUDA"):
        kps.token_logprobs(x.requires_grad_(), t)


def test_reference_against_definitions_and_differences():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(6, 19, dtype=torch.float64, generator=g) * 3
    tokens = torch.tensor([0, 5, 18, 7, -1, 3])
    x[1, 5] = x[1].max() + 1.0  # a token that is its row's largest
    x[2, 4] = -math.inf
    T = torch.tensor([1.0, 0.7, 2.0, 1.0, 1.0, 1.3])
    up, down = torch.randn(6, generator=g), torch.randn(6, generator=g)

    def value(y):
        r = score_reference(y, tokens, 0, T)
        return r["logprob"], r["entropy"]

    logp = torch.log_softmax(x / T.double()[:, None], 1)
    lp, H = value(x)
    live = tokens >= 0
    assert torch.allclose(lp[live], logp.gather(1, tokens.clamp(min=0)[:, None])[live, 0])
    assert torch.allclose(H[live], torch.special.entr(logp.exp()).sum(1)[live])
    grad, _ = Rows(x, tokens, T).grad(up, down)
    h = 1e-5
    for v in range(19):
        d = torch.zeros_like(x)
        d[:, v] = h
        (a, b), (c, e) = value(x + d), value(x - d)
        diff = (up * (a - c) + down * (b - e)) / (2 * h)
        assert torch.allclose(diff, grad[:, v], atol=1e-8, rtol=0)


# ---- on the GPU ---------------------------------------------------------------------------------
gpu = pytest.mark.gpu


def check(x, tokens, n=0, temperature=1.0, got=None):
    import decode_token_sampling_gb300 as kps
    got = kps.token_logprobs(x, tokens, n, temperature=temperature) if got is None else got
    torch.cuda.synchronize()
    want = score_reference(x, tokens, n, temperature)
    assert torch.equal(got.rank, want["rank"])
    for name in ("logprob", "entropy") + (("logprobs",) if n else ()):
        close(getattr(got, name), want[name], want[name + "_tol"], name)
    if n:
        assert torch.equal(got.ids, want["ids"])
    else:
        assert got.ids is None and got.logprobs is None
    return got


def check_grad(x, tokens, g, h, temperature=1.0):
    import decode_token_sampling_gb300 as kps
    _, stats = kps.token_logprobs_forward(x, tokens, temperature=temperature)
    got = kps.token_logprobs_backward(g, h, x, tokens, stats, temperature=temperature)
    torch.cuda.synchronize()
    want, tol = Rows(x, tokens, temperature).grad(g, h)
    close_grad(got, want, tol)
    return got


def make(N, V, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, V, device="cuda", generator=g) * 2.5
    x += (4 + 12 * torch.rand(N, 1, device="cuda", generator=g)) / torch.sqrt(torch.rand(N, V, device="cuda", generator=g) * V + 1)
    x = x.to(dtype)
    tokens = torch.randint(0, V, (N,), device="cuda", generator=g)
    tokens[::2] = x[::2].argmax(1)
    return x, tokens


def upstream(N, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    return torch.randn(N, device="cuda", generator=g), 0.3 * torch.randn(N, device="cuda", generator=g)


DTYPES = [torch.float32, torch.bfloat16]
SIZES = [(1, 1, 1), (2, 1, 0), (3, 2, 2), (2, 7, 0), (2, 9, 3), (5, 31, 31), (4, 600, 600), (2, 1000, 0), (3, 2047, 5), (3, 2048, 1024),
         (3, 2049, 0), (2, 4097, 1), (7, 4096, 700), (300, 5003, 20), (301, 5003, 0), (1, 32000, 20), (5, 32000, 0), (2, 50001, 1000),
         (1, 151936, 20), (1, 151936, 0), (160, 20001, 64), (200, 40001, 20), (300, 33000, 5), (2, 262144, 1024), (1, 1 << 20, 100), (2, 300001, 0), (1, 1 << 20, 0)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V,n", SIZES)
def test_sizes(N, V, n, dtype):
    x, tokens = make(N, V, dtype, seed=V + n)
    check(x, tokens, n)
    g, h = upstream(N)
    check_grad(x, tokens, g, h)
    tokens[0] = V
    check(x, tokens, n, 0.7)
    check_grad(x, tokens, g, h, 0.7)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 17])
def test_strides_and_offsets(dtype, n):
    for N, V, ld, off in ((6, 1001, 1024, 0), (6, 5001, 5027, 3), (9, 4097, 4097, 1), (5, 9000, 9008, 8), (1, 5000, 6000, 5), (400, 1999, 2003, 7)):
        buf = torch.full((N * ld + 64,), math.nan, dtype=dtype, device="cuda")
        view = buf[off:off + N * ld].view(N, ld)[:, :V]
        x, tokens = make(N, V, dtype, seed=ld)
        view.copy_(x)
        tokens[0] = 0
        tokens[-1] = V - 1
        check(view, tokens, n, 2.0)
        check_grad(view, tokens, *upstream(N), 2.0)


def _hard_rows(dtype, V, seed):
    """Rows of ties, masks, spikes, few finite tokens, infinities and NaN."""
    x, _ = make(20, V, dtype, seed=seed)
    low = torch.finfo(dtype).min
    at = torch.randperm(V, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    x[0] = 1.5
    x[1] = torch.randint(0, 3, (V,), device="cuda").to(dtype)
    x[2] = -math.inf
    x[2, at[:300]] = x[3, at[:300]]  # a vocabulary mask: 300 tokens allowed
    x[3] = low
    x[3, at[:600]] = x[4, at[:600]]  # the same with the type's lowest value
    x[4] = -1e4
    x[4, at[:30]] = x[5, at[:30]]
    x[5] = -math.inf
    x[6, at[:50]] += 200.0
    x[7, at[:min(V // 8, 5000)]] = 30.0  # a plateau longer than a list
    x[8, at[:3]] = math.nan
    x[9] = math.nan
    x[10, at[:2]] = math.inf
    x[11] = -math.inf
    x[11, at[0]] = 3.0
    x[12] = torch.arange(V, device="cuda").to(dtype) / 100  # ascending: every round has a new largest
    x[13] = -torch.arange(V, device="cuda").to(dtype) / 100
    x[14] = x[14] * 0
    x[14, ::2] = -x[14, ::2]  # zeros of both signs are equal
    x[15] = x[15] - 1e9 if dtype == torch.float32 else x[15] * 100
    x[16] = low  # uniform over the lowest value
    x[17] = low
    x[17, ::2] = -math.inf
    x[18, at[:1]] = 300.0  # certain
    x[19] = x[19] * 1e30
    return x, at


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 1, 20, 500])
@pytest.mark.parametrize("V", [1021, 40000])
def test_hard_rows(n, V, dtype):
    x, at = _hard_rows(dtype, V, n)
    N = len(x)
    top = torch.where(torch.isnan(x), -math.inf, x).argmax(1)
    g, h = upstream(N)
    for tokens in (at[:N], top, torch.full((N,), V - 1, device="cuda"), at[:1].expand(N).contiguous()):
        check(x, tokens, n)
        check(x, tokens, n, 0.25)
        check_grad(x, tokens, g, h)
        check_grad(x, tokens, g, h, 0.25)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 5, 20, 31, 32, 33])
@pytest.mark.parametrize("copies,V", [(1, 1000), (1, 50003), (1, 151936), (20, 40009), (40, 20011)])
def test_alternatives_of_rows_that_bounds_misjudge(n, copies, V, dtype):
    """Vocabularies in order, plateaus that begin late, masks with fewer tokens than alternatives, the largest
    logits in few of a warp's lanes."""
    low = torch.finfo(dtype).min
    x, _ = make(12, V, dtype, seed=V + n)
    at = torch.randperm(V, device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    i = torch.arange(V, device="cuda")
    x[0] = (i * (60.0 / V)).to(dtype)
    x[1] = (-i * (60.0 / V)).to(dtype)
    x[2] = 0.0
    x[2, V // 2:] = 1.0
    x[3] = -math.inf
    x[3, at[:7]] = x[4, at[:7]]
    x[4] = low
    x[4, at[:7]] = x[5, at[:7]]
    x[5] = -math.inf
    x[5, at[:300]] = x[6, at[:300]]
    x[6] = low
    x[6, at[:300]] = x[7, at[:300]]
    x[7] = torch.where(i // (8 if dtype == torch.bfloat16 else 4) % 32 < 3, 30.0 + x[7].float(), x[7].float()).to(dtype)
    x[8, at[:3]] = math.nan
    x[9] = (i % 977).to(dtype)  # values in cycles, each many times
    x[10] = -math.inf
    x[10, at[0]] = 3.0
    x[11, V // 3:] += 20.0
    x = x.repeat(copies, 1)
    tokens = at[:1].expand(len(x)).contiguous()
    check(x, tokens, n)


@gpu
@pytest.mark.parametrize("n", [0, 3])
@pytest.mark.parametrize("N", [1, 500])
def test_hard_rows_of_long_vocabularies(n, N):
    """A row shared by a cluster's CTAs, parts of which hold nothing, and whole rows."""
    V = 151936
    x = torch.full((N, V), -math.inf, device="cuda", dtype=torch.bfloat16)
    x[:, V - 3:] = torch.tensor([1.0, 2.0, 2.0], device="cuda", dtype=torch.bfloat16)
    tokens = torch.full((N,), V - 3, device="cuda")
    check(x, tokens, n)
    x[:, 5] = 2.0
    check(x, tokens, n)
    check_grad(x, tokens, *upstream(N))
    x[:, 70000] = math.nan
    check(x, tokens, n)
    x[:, 70000] = math.inf
    check(x, tokens, n)
    x.zero_()
    check(x, tokens, n)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 4])
def test_nearly_certain_rows_keep_their_relative_precision(dtype, n):
    """Logits whose differences are exact: entropies and log-probabilities from 1 to 1e-25, each to its own size."""
    gaps = [0, 1, 2, 4, 8, 12, 16, 20, 24, 32, 40, 50, 56]
    for V in (100, 5000, 100001):
        x = torch.zeros(len(gaps), V, device="cuda", dtype=dtype)
        x[:, V // 3] = torch.tensor(gaps, device="cuda", dtype=dtype)
        tokens = torch.full((len(gaps),), V // 3, device="cuda")
        got = check(x, tokens, n)
        want = score_reference(x, tokens, n)
        for name in ("logprob", "entropy"):
            # a sum right to a few 1e-5 (its additions by 256 threads, bounded in turn), not to 2^-24 of 1
            rel = (getattr(got, name).double() / want[name] - 1).abs()
            assert bool((rel <= 1e-4).all()), (name, rel)
        g, h = torch.ones(len(gaps), device="cuda"), torch.zeros(len(gaps), device="cuda")
        grad = check_grad(x, tokens, g, h)[:, V // 3].double()
        true = -torch.expm1(want["logprob"])
        assert bool(((grad / true - 1).abs() <= 1e-4 + torch.finfo(dtype).eps / 2).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [0, 5])
def test_temperatures_per_row(dtype, n):
    """Those of the sampling step: its greedy rows count as 1."""
    for V in (777, 30001):
        T = torch.tensor([1.0, 0.5, 1.7, 0.0, -1.0, math.nan, math.inf, -math.inf, 1e-39, 1.2e-38, 1e-3, 50.0, 1e10, 3e38], device="cuda")
        x, tokens = make(len(T), V, dtype, seed=9)
        check(x, tokens, n, T)
        check_grad(x, tokens, *upstream(len(T)), T)
        one = check(x, tokens, n, 1.0)
        row = check(x, tokens, n, torch.ones_like(T))
        assert all(torch.equal(a, b) for a, b in zip(one, row) if a is not None)


@gpu
@pytest.mark.parametrize("n", [0, 3])
def test_empty_rows_are_not_read(n):
    import decode_token_sampling_gb300 as kps
    for N, V in ((6, 1000), (6, 100000), (700, 5000)):
        x, tokens = make(N, V)
        dead = torch.arange(N, device="cuda") % 3 == 1
        x[dead] = math.nan
        tokens[dead] = torch.where(torch.arange(N, device="cuda") % 2 == 0, -100, V)[dead]
        got = check(x, tokens, n)
        assert bool((got.rank[dead] == -1).all()) and bool((got.entropy[dead] == 0).all())
        g, h = upstream(N)
        grad = check_grad(x, tokens, g, h)
        assert bool((grad[dead] == 0).all())
        # rows whose factors are both 0 neither
        live = torch.where(dead, 0, tokens)
        g[dead] = h[dead] = 0
        x[dead] = math.nan
        _, stats = kps.token_logprobs_forward(x, live)
        assert bool((kps.token_logprobs_backward(g, h, x, live, stats)[dead] == 0).all())
        assert bool((kps.token_logprobs_backward(None, None, x, live, stats) == 0).all())


@gpu
def test_no_rows():
    import decode_token_sampling_gb300 as kps
    x, tokens = make(3, 100)
    got = kps.token_logprobs(x[:0], tokens[:0], 5)
    assert got.logprob.shape == (0,) and got.ids.shape == (0, 5)
    x = x[:0].requires_grad_()
    t = kps.token_logprobs(x, tokens[:0])
    grad, = torch.autograd.grad(t.logprob.sum() + t.entropy.sum(), x)
    assert grad.shape == (0, 100)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_autograd(dtype):
    import decode_token_sampling_gb300 as kps
    x, tokens = make(9, 3001, dtype)
    tokens[4] = -100
    T = torch.rand(9, device="cuda") + 0.5
    g, h = upstream(9)
    leaf = x.clone().requires_grad_()
    for gg, hh in ((g, h), (g, None), (None, h)):
        t = kps.token_logprobs(leaf, tokens, 4, temperature=T)
        check(x, tokens, 4, T, got=kps.TokenLogprobs(*(v.detach() for v in t)))
        assert not t.rank.requires_grad and not t.ids.requires_grad and not t.logprobs.requires_grad
        outs = [(o, u) for o, u in ((t.logprob, gg), (t.entropy, hh)) if u is not None]
        grad, = torch.autograd.grad([o for o, _ in outs], leaf, [u for _, u in outs])
        want, tol = Rows(x, tokens, T).grad(gg, hh)
        close_grad(grad, want, tol)
    # a broadcast upstream gradient, a leaf used twice, a mean over a view
    t = kps.token_logprobs(leaf, tokens)
    (t.logprob.sum() + kps.token_logprobs(leaf, tokens).entropy.mean()).backward()
    one = torch.ones(9, device="cuda")
    a, at = Rows(x, tokens).grad(one, None)
    b, bt = Rows(x, tokens).grad(None, one / 9)
    half = torch.finfo(dtype).eps / 2
    close_grad(leaf.grad, a + b, (at + bt) * (1 + 2 * half) + half * (a.abs() + b.abs()) + 1e-40)
    with torch.no_grad():
        assert not kps.token_logprobs(leaf, tokens).logprob.requires_grad
    with pytest.raises(RuntimeError):
        u, = torch.autograd.grad(kps.token_logprobs(leaf, tokens).logprob.sum(), leaf, create_graph=True)
        u.sum().backward()


@gpu
def test_against_differences_of_the_kernel_itself():
    """Steps of 2^-4 on exactly representable logits: central differences are off by h^2 / 6 of a third
    derivative (below 1 for a log-probability, below 8 for an entropy of 25 tokens), and by the values'
    roundings over h."""
    import decode_token_sampling_gb300 as kps
    x = (torch.randn(4, 25, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) * 64).round() / 64
    tokens = torch.tensor([0, 7, 24, 3], device="cuda")
    g, h = upstream(4)
    grad = check_grad(x, tokens, g, h, 1.0)
    step = 2.0 ** -4
    for v in range(25):
        d = torch.zeros_like(x)
        d[:, v] = step
        a, b = kps.token_logprobs(x + d, tokens), kps.token_logprobs(x - d, tokens)
        diff = (g * (a.logprob - b.logprob) + h * (a.entropy - b.entropy)) / (2 * step)
        bound = step ** 2 / 6 * (g.abs() + 8 * h.abs()) + 1e-4
        assert bool(((diff - grad[:, v]).abs() <= bound).all())


@gpu
@pytest.mark.parametrize("n", [0, 30, 200])
def test_streams_graphs_and_repetition(n):
    import decode_token_sampling_gb300 as kps
    x, tokens = make(20, 32000, torch.bfloat16)
    g, h = upstream(20)
    want = check(x, tokens, n)
    want_grad = kps.token_logprobs_backward(g, h, x, tokens, kps.token_logprobs_forward(x, tokens, n)[1])
    close_grad(want_grad, *Rows(x, tokens).grad(g, h))
    side = torch.cuda.Stream()
    runs, grads = [], []
    for stream in (side, None, side):
        out, stats = kps.token_logprobs_forward(x, tokens, n, stream=stream)
        runs.append(out)
        grads.append(kps.token_logprobs_backward(g, h, x, tokens, stats, stream=stream))
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    y, ty = torch.zeros_like(x), torch.zeros_like(tokens)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, stats = kps.token_logprobs_forward(y, ty, n)
        runs.append(out)
        grads.append(kps.token_logprobs_backward(g, h, y, ty, stats))
        leaf = y.detach().requires_grad_()
        t = kps.token_logprobs(leaf, ty, n)
        auto, = torch.autograd.grad([t.logprob, t.entropy], leaf, [g, h])
        grads.append(auto)
    for _ in range(2):
        y.copy_(x)
        ty.copy_(tokens)
        graph.replay()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
    assert all(torch.equal(a, want_grad) for a in grads)


@gpu
@pytest.mark.parametrize("n", [0, 2, 40])
def test_many_short_rows(n):
    """More rows than a grid's other dimensions could hold; the same bits from call to call."""
    for N, V in ((70001, 3 if n < 40 else 50), (2000, 4003)):
        x, tokens = make(N, V, torch.bfloat16, seed=n)
        m = min(n, V)
        one, two = check(x, tokens, m), check(x, tokens, m)
        assert all(torch.equal(a, b) for a, b in zip(one, two) if a is not None)
        check_grad(x, tokens, *upstream(N))


@gpu
def test_two_host_threads():
    import threading
    import decode_token_sampling_gb300 as kps
    cases = [make(30, 20011, torch.bfloat16, seed=i) for i in range(2)]
    g, h = upstream(30)

    def job(x, tokens):
        t, stats = kps.token_logprobs_forward(x, tokens, 25)
        leaf = x.clone().requires_grad_()
        r = kps.token_logprobs(leaf, tokens)
        grad, = torch.autograd.grad([r.logprob, r.entropy], leaf, [g, h])
        p = kps.policy_loss_grad(x, tokens, g, h)
        return [*t, kps.token_logprobs_backward(g, h, x, tokens, stats), grad, *p]

    want = [job(*c) for c in cases]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(job(*cases[i]))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


@gpu
def test_logits_changed_before_the_backward_are_refused():
    import decode_token_sampling_gb300 as kps
    x, tokens = make(3, 100)
    leaf = x.clone().requires_grad_()
    y = leaf * 1.0
    t = kps.token_logprobs(y, tokens)
    with torch.no_grad():
        y.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        t.logprob.sum().backward()


@gpu
def test_more_than_2_to_31_elements():
    import decode_token_sampling_gb300 as kps
    N, V = 15000, 151936
    big = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_()
    tokens = torch.randint(0, V, (N,), device="cuda")
    rows = torch.tensor([0, 14133, 14134, 14135, N - 1], device="cuda")
    for n in (0, 10):
        got, stats = kps.token_logprobs_forward(big, tokens, n)
        check(big[rows], tokens[rows], n, got=kps.TokenLogprobs(*(None if v is None else v[rows] for v in got)))
    g, h = upstream(N)
    grad = kps.token_logprobs_backward(g, h, big, tokens, stats)
    want, tol = Rows(big[rows], tokens[rows]).grad(g[rows], h[rows])
    close_grad(grad[rows], want, tol)


@gpu
def test_outputs_that_are_not_wanted():
    import decode_token_sampling_gb300 as kps
    lib = kps.load_library()
    x, tokens = make(3, 5000)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for n in (0, 7):
        want = check(x, tokens, n)
        fields = [(3,), (3,), (3,), (3, 7), (3, 7), (9,)]
        kinds = [torch.float32, torch.float32, torch.int32, torch.int32, torch.float32, torch.float32]
        for mask in ((1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (0, 0, 0, 0)):
            wanted = [mask[0], mask[1], mask[2], n > 0, n > 0, mask[3]]
            bufs = [torch.full((math.prod(f) + 5,), -5, dtype=k, device="cuda") for f, k in zip(fields, kinds)]
            assert lib.kps_token_logprobs(p(x), 0, 3, 5000, 5000, p(tokens), n, 1.0, None, *(p(b) if w else None for b, w in zip(bufs, wanted)), s) == 0
            torch.cuda.synchronize()
            for b, w, f, v in zip(bufs, wanted, fields, want):
                size = math.prod(f) if w else 0
                assert bool((b[size:] == -5).all())  # nothing behind the last row
                if w and v is not None:
                    assert torch.equal(b[:size].view(f), v)


@gpu
def test_binding_refusals():
    import decode_token_sampling_gb300 as kps
    x, tokens = make(4, 100)
    T = torch.ones(4, device="cuda")
    for bad in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.t()), dict(logits=x[:1].expand(4, 100)), dict(n=101), dict(n=-1),
                dict(tokens=tokens.int()), dict(tokens=tokens.cpu()), dict(tokens=None), dict(tokens=tokens[:3]), dict(tokens=tokens[:, None]),
                dict(temperature=T.double()), dict(temperature=T[:3]), dict(temperature=T.cpu()),
                dict(temperature=T.clone().requires_grad_()), dict(logits=x.clone().requires_grad_(), stream=torch.cuda.Stream())):
        kw = dict(logits=x, tokens=tokens, n=5)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kps.token_logprobs(**kw)
    for bad in (0.0, -1.0, math.nan, math.inf):
        with pytest.raises(kps.KpsError):
            kps.token_logprobs(x, tokens, temperature=bad)
    _, stats = kps.token_logprobs_forward(x, tokens)
    one = torch.ones(4, device="cuda")
    for args in ((one.double(), None, x, tokens, stats), (None, one[:3], x, tokens, stats), (one, one, x, tokens, stats.t()),
                 (one, one, x, tokens, stats[:2]), (one, one, x, tokens, None)):
        with pytest.raises((TypeError, ValueError)):
            kps.token_logprobs_backward(*args)


@gpu
def test_after_the_sampling_step():
    """As serving uses it: tokens sampled at temperatures of their own, scored at the same ones."""
    import decode_token_sampling_gb300 as kps
    x, _ = make(70, 32000, torch.bfloat16, seed=4)
    T = torch.rand(70, device="cuda") + 0.5
    T[3] = 0.0  # greedy
    k = torch.full((70,), 40, dtype=torch.int32, device="cuda")
    idx, _ = kps.sample(x, k, torch.full((70,), 0.95, device="cuda"), T, None, seed=3)
    got = check(x, idx, 20, T)
    assert bool((got.rank < 40).all()) and int(got.rank[3]) == 0
    # the token is among the alternatives at its rank (unless an equal logit stands there)
    top = kps.top_logits(x, 20)
    assert torch.equal(got.ids, top.ids)
    inside = got.rank < 20
    assert bool((got.logprobs[inside].gather(1, got.rank[inside].long()[:, None])[:, 0] == got.logprob[inside]).all())
