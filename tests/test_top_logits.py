"""The top logits of a row with their log-sum-exps (kps_top_logits) against a 64-bit form."""

import ctypes
import math

import pytest
import torch

from logits_reference import EX2, U, sum_error, top_reference

FAKE = ctypes.c_void_p(1 << 20)


@pytest.fixture(scope="module")
def lib():
    from decode_token_sampling_gb300 import build
    build.build()
    import decode_token_sampling_gb300 as kps
    return kps.load_library()


def _call(lib, **over):
    args = dict(logits=FAKE, dt=0, B=4, V=100, ld=100, n=8, tau=1.0, tokens=None, ids=FAKE, values=FAKE, lse=FAKE,
                rest=FAKE, logprob=None, stream=None)
    args.update(over)
    return lib.kps_top_logits(*args.values())


def test_refusals(lib):
    for bad in (dict(dt=2), dict(B=-1), dict(V=0), dict(ld=99), dict(n=-1), dict(n=101), dict(n=1025, V=5000, ld=5000),
                dict(tau=0.0), dict(tau=-2.0), dict(tau=math.nan), dict(tau=math.inf), dict(tau=1e-40), dict(logits=None),
                dict(ids=None), dict(values=None), dict(logprob=FAKE), dict(logits=ctypes.c_void_p((1 << 20) + 2)),
                dict(ids=ctypes.c_void_p((1 << 20) + 2)), dict(tokens=ctypes.c_void_p((1 << 20) + 4), logprob=FAKE)):
        assert _call(lib, **bad) == 1, bad
    assert _call(lib, V=(1 << 20) + 1, ld=1 << 21) == 2
    assert _call(lib, B=1 << 40) == 2
    assert _call(lib, B=0, logits=None) == 0
    if not torch.cuda.is_available():
        assert _call(lib) == 4
        assert _call(lib, n=0, ids=None, values=None, lse=None, rest=None) == 4


def test_binding_refuses_cpu_tensors():
    import decode_token_sampling_gb300 as kps
    with pytest.raises(ValueError, match="CUDA"):
        kps.top_logits(torch.zeros(2, 10), 3)


gpu = pytest.mark.gpu


def check(x, n, tau=1.0, tokens=None, **kw):
    import decode_token_sampling_gb300 as kps
    got = kps.top_logits(x, n, temperature=tau, tokens=tokens, **kw)
    torch.cuda.synchronize()
    want = top_reference(x, n, tau, tokens)
    assert torch.equal(got.ids, want["ids"])
    assert torch.equal(got.values.double(), want["values"])
    # ln of a sum off by sum_error, the list's part of it added in up to 16 turns a thread; the
    # exponents' own errors; the reference divided by tau and the final addition
    d = 2 * sum_error(x.shape[1], x.dtype == torch.bfloat16) + 16 * U
    for name in ("lse", "rest"):
        w = want[name]
        _close(getattr(got, name).double(), w, d + 3 * U * 90 + 4 * U * w.abs(), name)
    if tokens is not None:
        w = want["logprob"]
        _close(got.logprob.double(), w, d + 3 * U * 90 + 4 * U * (w.abs() + 90), "logprob")
    else:
        assert got.logprob is None
    return got


def _close(got, want, tol, what):
    special = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(same[special].all()), f"{what}: NaN or inf differ"
    off = (got - want).abs()[~special]
    assert bool((off <= tol.expand_as(want)[~special]).all()), f"{what}: off by {float(off.max()):.3g}"


def _logits(B, V, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, V, device="cuda", generator=g) * 2.5
    x += 10 / torch.sqrt(torch.rand(B, V, device="cuda", generator=g) * V + 1)
    return x.to(dtype)


SIZES = [(1, 1, 1), (1, 1, 0), (3, 2, 2), (2, 7, 3), (5, 31, 31), (4, 600, 600), (2, 1000, 1000), (3, 2047, 5), (3, 2048, 1024),
         (3, 2049, 1024), (2, 4097, 1), (7, 4096, 700), (300, 5003, 20), (1, 32000, 20), (5, 32000, 0), (2, 50001, 1000),
         (1, 151936, 20), (1, 151936, 1024), (160, 20001, 64), (2, 262144, 1024), (1, 1 << 20, 100), (2, 300001, 1)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,n", SIZES)
def test_sizes(B, V, n, dtype):
    x = _logits(B, V, dtype, seed=V + n)
    tokens = torch.randint(0, V, (B,), device="cuda")
    check(x, n, 1.0, tokens)
    tokens[0] = V
    check(x, n, 0.7, tokens)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_offsets(dtype):
    for B, V, ld, off in ((6, 1001, 1024, 0), (6, 5001, 5027, 3), (9, 4097, 4097, 1), (5, 9000, 9008, 8), (1, 5000, 6000, 5)):
        buf = torch.full((B * ld + 64,), math.nan, dtype=dtype, device="cuda")
        view = buf[off:off + B * ld].view(B, ld)[:, :V]
        view.copy_(_logits(B, V, dtype, seed=ld))
        check(view, 17, 2.0)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 20, 500])
def test_rows_that_a_sample_misjudges(n, dtype):
    """Ties, constants, masks, spikes beside the sampled places, few finite tokens, infinities, NaN."""
    V = 40000
    x = _logits(16, V, dtype, seed=n)
    at = torch.randperm(V, device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    x[0] = 1.5
    x[1] = torch.randint(0, 3, (V,), device="cuda").to(dtype)
    x[2] = -math.inf
    x[2, at[:300]] = x[3, at[:300]]  # a vocabulary mask: 300 tokens allowed
    x[3] = torch.finfo(dtype).min
    x[3, at[:600]] = x[4, at[:600]]  # the same with the type's lowest value
    x[4] = -1e4
    x[4, at[:30]] = x[5, at[:30]]
    x[5] = -math.inf
    x[6, at[:50]] += 200.0  # a rest far below the top
    x[7, at[:5000]] = 30.0  # a plateau longer than the list
    x[8, at[:3]] = math.nan
    x[9] = math.nan
    x[10, at[:2]] = math.inf
    x[11] = -math.inf
    x[11, at[0]] = 3.0
    x[12] = torch.arange(V, device="cuda").to(dtype) / 100  # sorted: the top is one end of the row
    x[13] = -torch.arange(V, device="cuda").to(dtype) / 100
    x[14] = x[14] * 0
    x[14, ::2] = -x[14, ::2]  # zeros of both signs are equal
    x[15] = x[15] - 1e9 if dtype == torch.float32 else x[15] * 100
    check(x, n, 1.0, at[:16])
    check(x[6:8], n, 0.25)


@gpu
def test_the_list_overflows_in_a_shared_row():
    """One row shared by a cluster's CTAs: too few and too many listed elements."""
    V = 151936
    x = torch.zeros(1, V, device="cuda")
    check(x, 50)
    x[0, V // 2:] = 1.0
    check(x, 1024)
    x = _logits(1, V, torch.float32)
    x[0, V - 5000:] += 50.0
    check(x, 1000)
    x[0, 3] = math.nan
    check(x, 1000)


@gpu
def test_streams_graphs_and_repetition():
    import decode_token_sampling_gb300 as kps
    x = _logits(20, 32000, torch.bfloat16)
    tokens = torch.randint(0, 32000, (20,), device="cuda")
    want = check(x, 30, 1.0, tokens)
    side = torch.cuda.Stream()
    runs = []
    for _ in range(3):
        runs.append(kps.top_logits(x, 30, tokens=tokens, stream=side))
        runs.append(kps.top_logits(x, 30, tokens=tokens))
    graph = torch.cuda.CUDAGraph()
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        runs.append(kps.top_logits(y, 30, tokens=tokens))
    y.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for got in runs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_more_than_2_to_31_elements():
    B, V = 15000, 151936
    big = torch.empty(B, V, dtype=torch.bfloat16, device="cuda").normal_()
    import decode_token_sampling_gb300 as kps
    got = kps.top_logits(big, 10)
    rows = torch.tensor([0, 14133, 14134, 14135, B - 1], device="cuda")
    want = top_reference(big[rows], 10, 1.0)
    assert torch.equal(got.ids[rows], want["ids"]) and torch.equal(got.values[rows].double(), want["values"])


@gpu
def test_outputs_that_are_not_wanted():
    import decode_token_sampling_gb300 as kps
    x = _logits(3, 5000, torch.float32)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    ids = torch.full((4, 7), -5, dtype=torch.int32, device="cuda")
    val = torch.full((4, 7), -5.0, device="cuda")
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert kps.load_library().kps_top_logits(p(x), 0, 3, 5000, 5000, 7, 1.0, None, p(ids), p(val), None, None, None, s) == 0
    want = top_reference(x, 7, 1.0)
    assert torch.equal(ids[:3], want["ids"]) and bool((ids[3] == -5).all()) and bool((val[3] == -5).all())


@gpu
def test_binding_refusals():
    import decode_token_sampling_gb300 as kps
    x = _logits(4, 100, torch.float32)
    for bad in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.t()), dict(logits=x[:1].expand(4, 100)), dict(n=101),
                dict(n=-1), dict(tokens=torch.zeros(4, dtype=torch.int32, device="cuda")), dict(tokens=torch.zeros(4, dtype=torch.int64)),
                dict(tokens=torch.zeros(5, dtype=torch.int64, device="cuda"))):
        kw = dict(logits=x, n=5)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kps.top_logits(**kw)
    with pytest.raises(kps.KpsError):
        kps.top_logits(x, 5, temperature=-1.0)
    assert kps.top_logits(x[:0], 5).ids.shape == (0, 5)


@gpu
def test_teacher_to_student():
    """The run as it is used: a teacher's row to its top logits, these to a student's loss and gradient,
    and the log-probability of a token sampled from the student."""
    import decode_token_sampling_gb300 as kps
    from logits_reference import distill_reference
    B, V, tau = 24, 32000, 2.0
    teacher, student = _logits(B, V, torch.bfloat16, 1), _logits(B, V, torch.bfloat16, 2)
    top = kps.top_logits(teacher, 50, temperature=tau)
    loss, grad = kps.distill_loss_grad(student, top.ids, top.values, temperature=tau, rest=top.rest)
    ref, ref_grad, tol, gtol = distill_reference(student, top.ids, top.values, tau, top.rest)
    assert bool(((loss.double() - ref).abs() <= tol).all())
    half = torch.finfo(torch.bfloat16).eps / 2
    assert bool(((grad.double() - ref_grad).abs() <= gtol * (1 + half) + half * ref_grad.abs()).all())
    # with the rest as one class the teacher's masses are those of its whole row
    full = torch.softmax(teacher.double() / tau, 1).gather(1, top.ids.long())
    mine = torch.exp(top.values.double() / tau - top.lse.double()[:, None])
    assert bool(((mine - full).abs() <= full * (2 * sum_error(V) + 8 * U * 30 + EX2)).all())
    one = lambda v: torch.full((B,), v, device="cuda")  # noqa: E731
    idx, _ = kps.sample(student.contiguous(), torch.full((B,), 40, dtype=torch.int32, device="cuda"), one(0.9), one(1.0), None, seed=5)
    got = kps.top_logits(student, 0, tokens=idx).logprob
    want = torch.log_softmax(student.double(), 1).gather(1, idx[:, None])[:, 0]
    assert bool(((got.double() - want).abs() <= 2 * sum_error(V) + 8 * U * 60).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [-100.0, -500.0, -1e4])
def test_listed_rows_far_below_zero(dtype, shift):
    """Rows whose sum is taken of listed elements alone (short ones, and masked ones with few finite
    tokens), far below zero: a log-probability of -12 at temperature 0.1 is an exponent of -120."""
    for V, n in ((5, 2), (100, 10), (1000, 10), (4096, 300), (4096, 0)):
        x = (_logits(4, V, torch.float32, seed=V) + shift).to(dtype)
        check(x, n, 1.0, torch.randint(0, V, (4,), device="cuda"))
    x = torch.log_softmax(_logits(4, 3000, torch.float32), 1).to(dtype)
    check(x, 20, 0.1, torch.randint(0, 3000, (4,), device="cuda"))
    # 40 allowed tokens of a long row, the others -inf or the type's lowest value
    V = 150001
    at = torch.randperm(V, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    x = torch.full((3, V), -math.inf, dtype=dtype, device="cuda")
    x[1] = torch.finfo(dtype).min
    x[:2, at[:40]] = (_logits(2, 40, torch.float32) + shift).to(dtype)
    x[2, at[:3]] = shift
    for n in (0, 1, 10, 39, 40, 41):
        check(x, n, 1.0, at[:3])


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 50001])
def test_logprob_where_the_log_sum_exp_overflows(dtype, V):
    """Rows of the type's lowest or largest value at a temperature below 1: the log-sum-exp leaves
    fp32, the token's log-probability does not.  It is -ln of the number of equal tokens."""
    import decode_token_sampling_gb300 as kps
    x = torch.full((4, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    x[1] = -x[1]
    x[2, ::2] = -math.inf
    x[3] = -x[3]
    x[3, ::2] = 0.0
    equal = torch.tensor([V, V, V // 2, V // 2], device="cuda")
    for n in (0, 5):
        got = kps.top_logits(x, n, temperature=0.5, tokens=torch.full((4,), 7, device="cuda"))
        want = -torch.log(equal.double())
        # the sum's error, ln's last place and the negation
        assert bool(((got.logprob.double() - want).abs() <= sum_error(V, dtype == torch.bfloat16) + 2 * U * 16).all())
        assert got.lse.tolist() == [-math.inf, math.inf, -math.inf, math.inf]
