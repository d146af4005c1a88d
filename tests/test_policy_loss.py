"""The clipped policy loss with its gradient (kps_policy_loss_grad) against its formula in 64 bits."""

import ctypes
import math

import pytest
import torch

from token_reference import close, close_grad, policy_reference

FAKE = ctypes.c_void_p(1 << 20)
OUT = ctypes.c_void_p(1 << 30)
odd = lambda by: ctypes.c_void_p((1 << 20) + by)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    from decode_token_sampling_gb300 import build
    build.build()
    import decode_token_sampling_gb300 as kps
    return kps.load_library()


def _call(lib, **over):
    args = dict(logits=FAKE, dt=0, N=4, V=100, ld=100, tokens=FAKE, tau=1.0, taus=None, old=FAKE, advantage=FAKE, ref=FAKE, weight=FAKE,
                lo=0.2, hi=0.2, kl=0.1, ent=0.1, loss=OUT, logprob=OUT, entropy=OUT, grad=OUT, ld_grad=100, stream=None)
    assert not set(over) - set(args)
    args.update(over)
    return lib.kps_policy_loss_grad(*args.values())


def test_refusals(lib):
    for bad in (dict(dt=2), dict(N=-1), dict(V=0), dict(ld=99), dict(tau=0.0), dict(tau=math.nan), dict(tau=math.inf), dict(tau=1e-40),
                dict(logits=None), dict(tokens=None), dict(logits=odd(2)), dict(tokens=odd(4)), dict(taus=odd(2)), dict(old=None),
                dict(advantage=None), dict(ref=None), dict(old=odd(2)), dict(advantage=odd(1)), dict(ref=odd(2)), dict(weight=odd(2)),
                dict(lo=-0.1), dict(hi=-0.1), dict(lo=math.nan), dict(hi=math.nan), dict(kl=math.inf), dict(kl=math.nan),
                dict(ent=math.inf), dict(ent=math.nan), dict(loss=None), dict(logprob=None), dict(entropy=None), dict(loss=odd(2)),
                dict(logprob=odd(2)), dict(entropy=odd(2)), dict(grad=None), dict(ld_grad=99), dict(grad=ctypes.c_void_p((1 << 30) + 2)),
                dict(grad=FAKE), dict(grad=ctypes.c_void_p((1 << 20) + 4 * 399)), dict(grad=ctypes.c_void_p((1 << 20) - 4 * 399))):
        assert _call(lib, **bad) == 1, bad
    assert _call(lib, V=(1 << 20) + 1, ld=1 << 21) == 2
    assert _call(lib, N=1 << 40) == 2
    assert _call(lib, N=0, logits=None, tokens=None, old=None) == 0
    if not torch.cuda.is_available():
        assert _call(lib) == 4
        assert _call(lib, kl=0.0, ref=None, weight=None, hi=math.inf, lo=math.inf) == 4


def test_binding_refuses_cpu_tensors():
    import decode_token_sampling_gb300 as kps
    one = torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        kps.policy_loss_grad(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int64), one, one)


def _case(N, V, dtype=torch.float32, dev="cuda", seed=0, empty=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(N, V, device=dev, generator=g) * 2.5
    x += (4 + 12 * torch.rand(N, 1, device=dev, generator=g)) / torch.sqrt(torch.rand(N, V, device=dev, generator=g) * V + 1)
    x = x.to(dtype)
    tokens = torch.randint(0, V, (N,), device=dev, generator=g)
    tokens[::2] = x[::2].argmax(1)
    lp = torch.log_softmax(x.double(), 1).gather(1, tokens[:, None])[:, 0]
    step = torch.randn(N, device=dev, generator=g) * 0.25
    for border in (math.log(0.8), math.log(1.2), math.log(1.28)):  # not within half a per cent of a clip's border
        step = torch.where((step - border).abs() < 0.005, step + 0.011, step)
    old = (lp - step).float()
    ref = (lp + 0.2 * torch.randn(N, device=dev, generator=g)).float()
    ref[::5] = lp[::5].float() + 1.5  # beyond the series
    A = torch.randn(N, device=dev, generator=g)
    A[::7] = 0.0
    w = torch.rand(N, device=dev, generator=g) + 0.5
    w[torch.randperm(N, device=dev, generator=g)[:empty // 2]] = 0.0
    tokens[torch.randperm(N, device=dev, generator=g)[:empty - empty // 2]] = -100
    return dict(logits=x, tokens=tokens, old=old, advantage=A, ref=ref, weight=w)


def test_reference_gradient_against_differences():
    s = _case(8, 23, torch.float64, "cpu", seed=3, empty=2)
    s["ref"][0] += 0.9

    def loss(x):
        return policy_reference(**dict(s, logits=x), clip=(0.2, 0.28), kl=0.1, ent=0.05, temperature=1.0)

    grad, h = loss(s["logits"])["grad"], 1e-5
    for v in range(23):
        d = torch.zeros_like(s["logits"])
        d[:, v] = h
        diff = (loss(s["logits"] + d)["loss"] - loss(s["logits"] - d)["loss"]) / (2 * h)
        assert torch.allclose(diff, grad[:, v], atol=1e-7, rtol=0)


# ---- on the GPU ---------------------------------------------------------------------------------
gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


def own(s, clip=(0.2, 0.28), kl=0.1, ent=0.05, temperature=1.0, **kw):
    import decode_token_sampling_gb300 as kps
    return kps.policy_loss_grad(s["logits"], s["tokens"], s["old"], s["advantage"], clip=clip, ref_logprob=s["ref"] if kl else None,
                                kl_coef=kl, entropy_coef=ent, weight=s["weight"], temperature=temperature, **kw)


def check(s, clip=(0.2, 0.28), kl=0.1, ent=0.05, temperature=1.0, got=None):
    got = own(s, clip, kl, ent, temperature) if got is None else got
    torch.cuda.synchronize()
    want = policy_reference(**s, clip=clip, kl=kl, ent=ent, temperature=temperature)
    for name in ("logprob", "entropy", "loss"):
        close(getattr(got, name), want[name], want[name + "_tol"], name)
    close_grad(got.grad, want["grad"], want["grad_tol"])
    return got


SIZES = [(1, 1), (3, 2), (2, 7), (5, 31), (4, 600), (3, 2048), (3, 2049), (7, 4097), (300, 5003), (5, 32000), (160, 20001), (1, 151936),
         (2, 262144), (1, 1 << 20), (40, 60000), (2, 500001)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V", SIZES)
def test_sizes(N, V, dtype):
    s = _case(N, V, dtype, seed=V, empty=N // 3)
    check(s)
    check(s, kl=0.0, ent=0.0)
    check(dict(s, weight=None), (0.1, 0.1), ent=0.0)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_offsets(dtype):
    for N, V, ld, off in ((6, 1001, 1024, 0), (6, 5001, 5027, 3), (9, 4097, 4097, 1), (5, 9000, 9008, 8), (1, 5000, 6000, 5), (400, 1999, 2003, 7),
                          (3, 60001, 60002, 1)):
        buf = torch.full((N * ld + 64,), math.nan, dtype=dtype, device="cuda")
        view = buf[off:off + N * ld].view(N, ld)[:, :V]
        s = _case(N, V, dtype, seed=ld)
        view.copy_(s["logits"])
        s["tokens"][0], s["tokens"][-1] = 0, V - 1
        s["old"] = torch.log_softmax(s["logits"].double(), 1).gather(1, s["tokens"][:, None])[:, 0].float() + 0.05
        check(dict(s, logits=view))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_gradient_of_another_phase(dtype):
    """The C ABI takes a gradient whose rows do not share the logits' 16-byte boundaries; what lies between its rows stays."""
    import decode_token_sampling_gb300 as kps
    lib = kps.load_library()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for N, V, ld in ((5, 5003, 5010), (2, 100001, 100003), (200, 1001, 1001)):
        s = _case(N, V, dtype, seed=V)
        out = torch.full((3, N), -5.0, device="cuda")
        buf = torch.full((N * ld + 9,), -5.0, dtype=dtype, device="cuda")
        code = 0 if dtype == torch.float32 else 1
        st = lib.kps_policy_loss_grad(p(s["logits"]), code, N, V, V, p(s["tokens"]), 1.0, None, p(s["old"]), p(s["advantage"]), p(s["ref"]),
                                      p(s["weight"]), 0.2, 0.28, 0.1, 0.05, p(out[0]), p(out[1]), p(out[2]), p(buf[3:]), ld,
                                      ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        rows = buf[3:3 + N * ld].view(N, ld)
        check(s, got=kps.PolicyLoss(out[0], rows[:, :V], out[1], out[2]))
        assert bool((buf[:3] == -5).all()) and bool((buf[3 + N * ld:] == -5).all()) and bool((rows[:, V:] == -5).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1021, 40000, 400001])
def test_hard_rows(V, dtype):
    s = _case(16, V, dtype, seed=V)
    x, low = s["logits"], torch.finfo(dtype).min
    x[0] = 1.5
    x[1] = torch.randint(0, 3, (V,), device="cuda").to(dtype)
    x[2] = -math.inf
    x[2, 100:400] = x[3, 100:400]
    x[3] = low
    x[3, 100:700] = x[4, 100:700]
    x[4] = -1e4
    x[5] = -math.inf
    x[6, :50] += 200.0
    x[7, V // 2:] = 30.0
    x[8, 3] = math.nan
    x[9] = math.nan
    x[10, V - 1] = math.inf
    x[11] = -math.inf
    x[11, 2] = 3.0
    x[12] = torch.arange(V, device="cuda").to(dtype) / 100
    x[13] = low
    x[13, ::2] = -math.inf
    x[14] = x[14] - 1e9 if dtype == torch.float32 else x[14] * 100
    x[15, V // 2] = 300.0
    finite = torch.where(torch.isnan(x) | (x == math.inf), -math.inf, x)
    top = finite.argmax(1)
    second = finite.scatter(1, top[:, None], -math.inf).argmax(1)
    for tokens, kl in ((top, 0.1), (second, 0.0)):  # (a token of probability 0 has an infinite penalty)
        lp = torch.log_softmax(x.double(), 1).gather(1, tokens[:, None])[:, 0]
        base = torch.where(torch.isfinite(lp), lp, 0.0).float()
        check(dict(s, tokens=tokens, old=base + 0.03, ref=base + 0.3), kl=kl)
        check(dict(s, tokens=tokens, old=base - 0.5, ref=base), kl=0.0, ent=-0.2)


@gpu
def test_ratios_at_their_extremes():
    """Tokens that the old policy gave far more or less, and advantages of 0 beside infinite ratios."""
    V = 5000
    s = _case(6, V, seed=5)
    lp = torch.log_softmax(s["logits"].double(), 1).gather(1, s["tokens"][:, None])[:, 0].float()
    s["old"] = lp + torch.tensor([-200.0, -200.0, -200.0, 200.0, 200.0, math.inf], device="cuda")
    s["advantage"] = torch.tensor([1.0, 0.0, 0.0, 1.0, -1.0, 0.5], device="cuda")
    got = check(s, kl=0.0)
    assert bool(torch.isfinite(got.loss).all()) and bool(torch.isfinite(got.grad).all())
    s["advantage"][1] = -1.0  # a ratio that leaves fp32 and is not clipped
    assert float(own(s, kl=0.0).loss[1]) == math.inf
    # no bounds
    s = _case(6, V, seed=6)
    check(s, (math.inf, math.inf))
    check(s, (0.0, 0.0))


@gpu
def test_small_penalties_keep_their_size():
    """exp(u) - u - 1 for u from 1 down to 2^-10: exact logits of two tokens, u an exact difference."""
    us = torch.tensor([2.0 ** -k for k in range(0, 11)] + [-(2.0 ** -k) for k in range(0, 11)], device="cuda")
    N = len(us)
    x = torch.full((N, 7), -math.inf, device="cuda")
    x[:, 3] = 1.0  # a certain token: log-probability 0
    tokens = torch.full((N,), 3, device="cuda")
    zero = torch.zeros(N, device="cuda")
    s = dict(logits=x, tokens=tokens, old=zero, advantage=zero, ref=us, weight=None)
    got = own(s, kl=1.0, ent=0.0)
    want = torch.expm1(us.double()) - us.double()
    # the product, the halving's factors and the series' nine steps, half a step each; beyond the series expm1's
    # 2 steps and the subtraction's, whose terms are at most 4 times the result at |u| >= 1/2
    assert bool(((got.loss.double() / want - 1).abs() <= 24 * 2.0 ** -24).all())
    assert bool((got.grad == 0).all())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_temperatures_per_row(dtype):
    T = torch.tensor([1.0, 0.5, 1.7, 0.0, -1.0, math.nan, math.inf, 1e-39, 0.8, 50.0], device="cuda")
    for V in (777, 60001):
        s = _case(len(T), V, dtype, seed=9)
        scale = torch.where((T >= 1.2e-38) & (T < math.inf), T, 1.0).double()
        lp = torch.log_softmax(s["logits"].double() / scale[:, None], 1).gather(1, s["tokens"][:, None])[:, 0].float()
        check(dict(s, old=lp + 0.07, ref=lp - 0.1), temperature=T)
    check(_case(9, 3001, dtype), temperature=1.0)


@gpu
@pytest.mark.parametrize("N,V", [(7, 1000), (7, 100000), (700, 5000), (6, 1 << 20)])
def test_empty_rows_are_not_read(N, V):
    s = _case(N, V)
    i = torch.arange(N, device="cuda")
    dead = i % 3 == 1
    s["logits"][dead] = math.nan
    s["weight"][dead & (i % 2 == 0)] = 0.0
    s["tokens"][dead & (i % 2 == 1)] = V
    got = check(s)
    for t in got:
        assert bool((t[dead] == 0).all())


@gpu
def test_no_rows():
    s = _case(3, 100)
    got = own({k: v[:0] for k, v in s.items()})
    assert got.loss.shape == (0,) and got.grad.shape == (0, 100)


@gpu
@pytest.mark.parametrize("N,V", [(20, 32000), (3, 700000)])
def test_streams_graphs_and_repetition(N, V):
    s = _case(N, V, torch.bfloat16, empty=3)
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
def test_more_than_2_to_31_elements():
    import decode_token_sampling_gb300 as kps
    N, V = 15000, 151936
    big = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_()
    s = dict(logits=big, tokens=torch.randint(0, V, (N,), device="cuda"), old=torch.full((N,), -12.0, device="cuda"),
             advantage=torch.ones(N, device="cuda"), ref=torch.full((N,), -12.5, device="cuda"), weight=torch.ones(N, device="cuda"))
    got = own(s, (0.9, 1e4))
    rows = torch.tensor([0, 14133, 14134, 14135, N - 1], device="cuda")
    check({k: v[rows] for k, v in s.items()}, (0.9, 1e4), got=kps.PolicyLoss(*(t[rows] for t in got)))


@gpu
def test_many_short_rows():
    s = _case(70001, 5, torch.bfloat16, seed=2, empty=1000)
    one, two = check(s), own(s)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@gpu
def test_a_token_of_probability_zero():
    """Without a penalty it has a ratio of 0; with one the loss is infinite, as its formula."""
    s = _case(4, 3000, seed=1)
    s["logits"][torch.arange(4), s["tokens"]] = -math.inf
    s["old"].fill_(-2.0)
    s["ref"].fill_(-2.0)
    s["advantage"] = torch.tensor([1.0, -1.0, 0.0, 2.0], device="cuda")
    got = check(s, kl=0.0)
    assert bool(torch.isfinite(got.loss).all()) and bool(torch.isfinite(got.grad).all())
    assert own(s, kl=0.1).loss.tolist() == [math.inf] * 4


@gpu
def test_binding_refusals():
    import decode_token_sampling_gb300 as kps
    s = _case(4, 100)
    for bad in (dict(logits=s["logits"].half()), dict(tokens=s["tokens"].int()), dict(old=s["old"].double()), dict(advantage=s["advantage"][:3]),
                dict(ref=s["ref"].cpu()), dict(weight=s["weight"][:, None]), dict(ref=None),
                dict(tokens=None), dict(old=None), dict(advantage=None)):
        with pytest.raises((TypeError, ValueError)):
            own(dict(s, **bad))
    for kw in (dict(clip=(-0.1, 0.2)), dict(clip=(0.2, math.nan)), dict(kl=math.inf), dict(ent=math.nan), dict(temperature=0.0)):
        with pytest.raises(kps.KpsError):
            own(s, **kw)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_the_run_of_a_training_step(dtype):
    """Tokens sampled from the old policy, its log-probabilities, a policy that has moved since: the loss and gradient in one
    call against the same loss of token_logprobs' outputs through autograd."""
    import decode_token_sampling_gb300 as kps
    N, V = 64, 20000
    s = _case(N, V, dtype, seed=8)
    one = torch.ones(N, device="cuda")
    old_logits = s["logits"]
    T = 0.9 * one
    tokens, _ = kps.sample(old_logits, torch.zeros(N, dtype=torch.int32, device="cuda"), one, T, None, seed=1)
    old = kps.token_logprobs(old_logits, tokens, temperature=T).logprob
    new = (old_logits.float() + 0.2 * torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(4))).to(dtype)
    A, w, ref = s["advantage"], s["weight"], old - 0.05
    fused = kps.policy_loss_grad(new, tokens, old, A, clip=(0.2, 0.28), ref_logprob=ref, kl_coef=0.05, entropy_coef=0.01, weight=w, temperature=T)
    leaf = new.clone().requires_grad_()
    t = kps.token_logprobs(leaf, tokens, temperature=T)
    ratio = torch.exp(t.logprob - old)
    loss = -torch.minimum(ratio * A, ratio.clamp(0.8, 1.28) * A)
    u = ref - t.logprob
    loss = w * (loss + 0.05 * (torch.exp(u) - u - 1) - 0.01 * t.entropy)
    grad, = torch.autograd.grad(loss.sum(), leaf)
    want = policy_reference(new, tokens, old, A, (0.2, 0.28), ref, 0.05, 0.01, w, T)
    away = ((torch.exp(want["logprob"] - old.double()) - 0.8).abs() > 1e-4) & ((torch.exp(want["logprob"] - old.double()) - 1.28).abs() > 1e-4)
    assert int(away.sum()) >= N - 2
    # both are within the bound of the same reference, autograd's loss with torch's exp and a plain exp(u) - u - 1
    # (half a step of 1 each, and of u) instead of the kernel's
    close(fused.loss[away], want["loss"][away], want["loss_tol"][away], "loss")
    close_grad(fused.grad[away], want["grad"][away], want["grad_tol"][away])
    slack = 2 * want["loss_tol"] + 8 * 2.0 ** -24 * w.double() * (1 + want["loss"].abs())
    close(loss.detach()[away], want["loss"][away], slack[away], "autograd's loss")
    close_grad(grad[away], want["grad"][away], (2 * want["grad_tol"] + 16 * 2.0 ** -24 * want["grad"].abs() + 1e-8)[away])
