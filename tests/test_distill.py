"""The distillation loss and its gradient (kps_distill_*) against the formulas in 64 bits."""

import ctypes
import math

import pytest
import torch

from logits_reference import U, distill_reference

FAKE = ctypes.c_void_p(1 << 20)


# ---- without a GPU: refusals, and the reference's own gradient against differences --------------

@pytest.fixture(scope="module")
def lib():
    from decode_token_sampling_gb300 import build
    build.build()
    import decode_token_sampling_gb300 as kps
    return kps.load_library()


def _forward(lib, **over):
    args = dict(student=FAKE, dt=0, N=4, V=100, ld=100, ids=FAKE, values=FAKE, values_dt=0, K=8, rest=None,
                weight=None, tau=1.0, loss=FAKE, stats=FAKE, stream=None)
    args.update(over)
    return lib.kps_distill_forward(*args.values())


def _loss_grad(lib, **over):
    args = dict(student=FAKE, dt=0, N=4, V=100, ld=100, ids=FAKE, values=FAKE, values_dt=0, K=8, rest=None,
                weight=None, tau=1.0, loss=FAKE, grad=ctypes.c_void_p(1 << 30), ld_grad=100, stream=None)
    args.update(over)
    return lib.kps_distill_loss_grad(*args.values())


def _backward(lib, **over):
    args = dict(student=FAKE, dt=0, N=4, V=100, ld=100, ids=FAKE, values=FAKE, values_dt=0, K=8, rest=None,
                weight=None, tau=1.0, grad_loss=None, stats=FAKE, grad=ctypes.c_void_p(1 << 30), ld_grad=100, stream=None)
    args.update(over)
    return lib.kps_distill_backward(*args.values())


@pytest.mark.parametrize("call", [_forward, _loss_grad, _backward])
def test_shared_refusals(lib, call):
    for bad in (dict(dt=2), dict(values_dt=7), dict(N=-1), dict(V=0), dict(K=0), dict(K=1025), dict(ld=99), dict(tau=0.0),
                dict(tau=-1.0), dict(tau=math.nan), dict(tau=math.inf), dict(tau=1e-39), dict(student=None),
                dict(ids=None), dict(values=None), dict(student=ctypes.c_void_p((1 << 20) + 2)),
                dict(ids=ctypes.c_void_p((1 << 20) + 2)), dict(rest=ctypes.c_void_p((1 << 20) + 1)),
                dict(weight=ctypes.c_void_p((1 << 20) + 3))):
        assert call(lib, **bad) == 1, bad
    assert call(lib, V=(1 << 20) + 1, ld=1 << 21) == 2
    assert call(lib, N=1 << 40) == 2
    assert call(lib, N=0, student=None) == 0  # a valid no-op


def test_own_refusals(lib):
    assert _forward(lib, loss=None) == 1
    assert _loss_grad(lib, loss=None) == 1
    assert _backward(lib, stats=None) == 1
    for call in (_loss_grad, _backward):
        assert call(lib, grad=None) == 1
        assert call(lib, ld_grad=99) == 1
        assert call(lib, grad=ctypes.c_void_p((1 << 30) + 2)) == 1
        # the student's own rows, and a buffer that overlaps their last or first element
        assert call(lib, grad=FAKE) == 1
        assert call(lib, grad=ctypes.c_void_p((1 << 20) + 4 * 399)) == 1
        assert call(lib, grad=ctypes.c_void_p((1 << 20) - 4 * 399)) == 1
    if not torch.cuda.is_available():  # valid calls: they fail only for want of a GPU
        assert _forward(lib, stats=None) == 4
        assert _loss_grad(lib, grad=ctypes.c_void_p((1 << 20) + 4 * 400)) == 4
        assert _backward(lib) == 4
        assert _backward(lib, N=1, ld=0, ld_grad=0) == 4  # one row has no row stride


def test_binding_refuses_cpu_tensors():
    import decode_token_sampling_gb300 as kps
    s, ids, val = torch.zeros(2, 10), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    for call in (kps.distill_loss, kps.distill_forward, kps.distill_loss_grad):
        with pytest.raises(ValueError, match="CUDA"):
            call(s, ids, val)
    with pytest.raises(ValueError, match="requires a gradient"):
        kps.distill_loss(s, ids, val.clone().requires_grad_())


def _case(N, V, K, dtype=torch.float32, dev="cpu", seed=0, rest=True, near=1.0, bonus=8.0):
    """A student near its teacher, the teacher's top K with the rest's log-sum-exp at tau 1."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    t = torch.randn(N, V, device=dev, generator=g) * 2
    t += bonus / torch.sqrt(torch.rand(N, V, device=dev, generator=g) * V + 1)
    s = (t + near * torch.randn(N, V, device=dev, generator=g)).to(dtype)
    values, ids = t.topk(min(K, V), dim=1)
    if K > V:  # more slots than tokens: the others are empty
        values = torch.cat([values, torch.zeros(N, K - V, device=dev)], 1)
        ids = torch.cat([ids, torch.full((N, K - V), -1, device=dev)], 1)
    r = None
    if rest:
        r = torch.logsumexp(t.scatter(1, ids.clamp(min=0), -math.inf), 1)
    return s, ids.to(torch.int32).contiguous(), values.contiguous(), r


def test_reference_gradient_against_differences():
    s, ids, val, rest = _case(5, 23, 6, torch.float64, seed=3)
    ids[0, 2] = ids[0, 1]  # the same token twice
    ids[1, 3:] = -1
    w = torch.tensor([1.0, 0.5, 0.0, 2.0, 1.0])
    tau, h = 1.5, 1e-5
    for r in (rest, None):
        loss, grad, _, _ = distill_reference(s, ids, val, tau, r, w)
        for v in range(23):
            d = torch.zeros_like(s)
            d[:, v] = h
            up, down = (distill_reference(s + e, ids, val, tau, r, w)[0] for e in (d, -d))
            # central differences: h^2 / 6 of a third derivative of order one, and 2^-52 |loss| / h
            assert torch.allclose((up - down) / (2 * h), grad[:, v], atol=1e-8, rtol=0)


# ---- on the GPU ---------------------------------------------------------------------------------

gpu = pytest.mark.gpu


def check(s, ids, val, tau=1.0, rest=None, weight=None, upstream=None):
    """Every entry point on the same inputs against the 64-bit formulas; returns (loss, grad)."""
    import decode_token_sampling_gb300 as kps
    kw = dict(temperature=tau, rest=rest, weight=weight)
    ref_loss, _, tol, _ = distill_reference(s, ids, val, tau, rest, weight)
    loss, stats = kps.distill_forward(s, ids, val, **kw)
    loss2, grad = kps.distill_loss_grad(s, ids, val, **kw)
    back = kps.distill_backward(upstream, s, ids, val, stats, **kw)
    for got in (loss, loss2):
        _compare(got.double(), ref_loss, tol, "loss")
    half = torch.finfo(s.dtype).eps / 2
    for got, up in ((grad, None), (back, upstream)):
        assert got.dtype == s.dtype and got.shape == s.shape
        _, ref, _, tol = distill_reference(s, ids, val, tau, rest, weight, up)
        _compare(got.double(), ref, tol + half * ref.abs() + half * tol, "grad")
    return loss, grad


def _compare(got, want, tol, what):
    special = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(same[special].all()), f"{what}: NaN or inf differ"
    off = (got - want).abs()[~special]
    lim = tol.expand_as(want)[~special]
    bad = ~(off <= lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / lim).max()):.3g} of the bound"


SIZES = [(1, 1, 1), (3, 2, 1), (2, 7, 9), (5, 31, 4), (1, 1000, 16), (37, 1000, 1), (4, 4099, 33), (2, 8195, 100),
         (7, 32000, 64), (300, 5003, 20), (3, 50001, 1024), (1, 151936, 64), (160, 8192, 8), (2, 262144, 40),
         (2, 450001, 33), (1, 1 << 20, 300)]  # rows that no cluster's shared memory holds among them


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,K", SIZES)
def test_sizes(N, V, K, dtype):
    for rest in (False, True):
        s, ids, val, r = _case(N, V, K, dtype, "cuda", seed=V + K, rest=rest)
        g = torch.rand(N, device="cuda") + 0.5
        check(s, ids, val, 1.0, r, None, g)
        check(s, ids, val.to(torch.bfloat16), 2.0, r, g, None)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_offsets(dtype):
    """Rows in a wider buffer, from an odd column on, and a batch whose row starts take every phase."""
    for N, V, ld, off in ((6, 1001, 1024, 0), (6, 1001, 1027, 3), (9, 4097, 4097, 1), (5, 2000, 2048, 8), (1, 5000, 6000, 5)):
        s, ids, val, r = _case(N, V, 20, dtype, "cuda", seed=ld)
        buf = torch.full((N * ld + 64,), math.nan, dtype=dtype, device="cuda")
        view = buf[off:off + N * ld].view(N, ld)[:, :V]
        view.copy_(s)
        check(view, ids, val, 0.7, r)
        check(view, ids, val, 0.7, None)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("phase", [0, 1, 5])
def test_gradient_buffer_of_the_callers(dtype, phase):
    """Any row stride and phase of the gradient; what lies outside its rows is left as it was."""
    import decode_token_sampling_gb300 as kps
    N, V, ld, ldg = 5, 3001, 3008, 3100
    s, ids, val, r = _case(N, V, 30, dtype, "cuda", seed=phase)
    weight = torch.tensor([1.0, 0.0, 2.0, 1.0, 0.5], device="cuda")
    buf = torch.zeros(N, ld, dtype=dtype, device="cuda")
    buf[:, :V] = s
    out = torch.full((N * ldg + 32,), 77.0, dtype=dtype, device="cuda")
    esize = out.element_size()
    loss = torch.empty(N, device="cuda")
    st = kps.load_library().kps_distill_loss_grad(
        ctypes.c_void_p(buf.data_ptr()), 1 if dtype == torch.bfloat16 else 0, N, V, ld, ctypes.c_void_p(ids.data_ptr()),
        ctypes.c_void_p(val.data_ptr()), 0, 30, ctypes.c_void_p(r.data_ptr()), ctypes.c_void_p(weight.data_ptr()), 1.0,
        ctypes.c_void_p(loss.data_ptr()), ctypes.c_void_p(out.data_ptr() + phase * esize), ldg,
        ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    _, ref, _, tol = distill_reference(s, ids, val, 1.0, r, weight)
    rows = out[phase:phase + N * ldg].view(N, ldg)
    half = torch.finfo(dtype).eps / 2
    _compare(rows[:, :V].double(), ref, tol + half * ref.abs() + half * tol, "grad")
    assert bool((rows[:, V:] == 77.0).all()) and bool((out[:phase] == 77.0).all()) and bool((out[phase + N * ldg:] == 77.0).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks(dtype):
    """Empty slots, empty rows, rows of weight 0 over NaN, masked student tokens."""
    s, ids, val, r = _case(12, 5000, 24, dtype, "cuda", seed=5)
    ids[0] = -1  # nothing in the list
    val[1] = -math.inf
    ids[2, 3:] = 5000  # outside the vocabulary
    val[3, 1] = -math.inf  # an empty slot by value: its token belongs to the rest
    ids[4, ::2] = -7
    weight = torch.ones(12, device="cuda")
    weight[5] = 0
    s[5] = math.nan
    s[0, 7] = math.nan
    weight[6] = 0
    s[6, 100] = math.inf
    listed = torch.zeros(5000, dtype=torch.bool, device="cuda")
    listed[ids[7].long()] = True
    s[7, ~listed & (torch.arange(5000, device="cuda") % 3 == 0)] = -math.inf
    s[8, :40] = torch.finfo(dtype).min  # the type's lowest value outside (mostly) of the list
    s[8, ids[8].long()] = torch.randn(24, device="cuda").to(dtype)
    s[9] = s[9] - 1e9 if dtype == torch.float32 else s[9]
    r[10] = -math.inf  # no rest in this row
    up = torch.ones(12, device="cuda")
    up[11] = 0
    for rest in (r, None):
        loss, grad = check(s, ids, val, 1.0, rest, weight, up)
        for row in (0, 1, 5, 6):
            assert float(loss[row]) == 0 and bool((grad[row] == 0).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_a_distribution(dtype):
    """NaN, +inf or nothing above -inf in the student's row: NaN; mass where the student has none: +inf."""
    s, ids, val, r = _case(6, 3000, 10, dtype, "cuda", seed=6)
    s[0, 17] = math.nan
    s[1, 2999] = math.inf
    s[2] = -math.inf
    s[3, ids[3, 0].long()] = -math.inf
    for rest in (r, None):
        loss, grad = check(s, ids, val, 1.0, rest)
        assert bool(torch.isnan(loss[:3]).all()) and bool(torch.isnan(grad[:3].float()).all())
        assert float(loss[3]) == math.inf
        assert bool(torch.isfinite(loss[4:]).all())
    # the list is the whole vocabulary, and the teacher's rest has mass all the same
    s, ids, val, _ = _case(2, 64, 64, dtype, "cuda", rest=False)
    import decode_token_sampling_gb300 as kps
    loss, _ = kps.distill_loss_grad(s, ids, val, rest=torch.zeros(2, device="cuda"))
    assert bool((loss == math.inf).all())
    check(s, ids, val, 1.0, torch.full((2,), -math.inf, device="cuda"))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0.0, 60.0, 150.0, 400.0, -400.0])
def test_student_far_from_its_list(dtype, shift):
    """The list's tokens lie far above or below everything else in the student's row."""
    s, ids, val, r = _case(4, 6000, 12, dtype, "cuda", seed=7)
    s.scatter_add_(1, ids.long(), torch.full((4, 12), shift, dtype=dtype, device="cuda"))
    for tau in (1.0, 0.25):
        check(s, ids, val, tau, r)
        check(s, ids, val, tau, None)
        check(s, ids, val, tau, r - 200.0)  # next to no mass outside the list
        check(s, ids, val, tau, r + 200.0)  # next to none in it


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_same_token_in_several_slots(dtype):
    s, ids, val, r = _case(40, 2000, 48, dtype, "cuda", seed=8)
    ids[0] = ids[0, 0]
    ids[1, 1::2] = ids[1, 0::2]
    ids[2, 10:13] = ids[2, 0]
    ids[3, 47] = ids[3, 0]
    ids[4:] = torch.randint(0, 40, (36, 48), device="cuda", dtype=torch.int32)
    runs = [check(s, ids, val, 1.3, rest) for rest in (r, None, r, None)]
    for a, b in ((0, 2), (1, 3)):  # the same bits each time
        assert torch.equal(runs[a][0], runs[b][0]) and torch.equal(runs[a][1], runs[b][1])


@gpu
def test_small_divergence_is_exact():
    """A student almost equal to its teacher: the loss is a small sum of terms that cancel."""
    for near, tau in ((0.05, 1.0), (0.01, 2.0)):
        s, ids, val, r = _case(20, 32000, 64, torch.float32, "cuda", seed=9, near=near, bonus=30.0)
        check(s, ids, val, tau, torch.logsumexp(s.double().scatter(1, ids.long(), -math.inf) / tau, 1).float())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_autograd(dtype):
    """Through autograd: a broadcast upstream gradient, a head in front, and differences of the loss."""
    import decode_token_sampling_gb300 as kps
    s, ids, val, r = _case(6, 4001, 16, dtype, "cuda", seed=10)
    leaf = s.clone().requires_grad_()
    kps.distill_loss(leaf, ids, val, temperature=2.0, rest=r).mean().backward()
    up = torch.full((6,), 1.0 / 6, device="cuda")
    _, ref, _, tol = distill_reference(s, ids, val, 2.0, r, None, up)
    half = torch.finfo(dtype).eps / 2
    _compare(leaf.grad.double(), ref, tol + half * ref.abs() + half * tol, "grad")
    h = torch.randn(6, 32, device="cuda", dtype=dtype)
    head = torch.randn(4001, 32, device="cuda", dtype=dtype, requires_grad=True)
    loss = kps.distill_loss(h @ head.t(), ids, val, temperature=2.0, rest=r)
    assert loss.requires_grad
    loss.sum().backward()
    assert head.grad.shape == head.shape and bool(torch.isfinite(head.grad.float()).all())
    with torch.no_grad():
        assert not kps.distill_loss(leaf, ids, val).requires_grad
    x = leaf.detach().requires_grad_()
    g, = torch.autograd.grad(kps.distill_loss(x, ids, val).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        torch.autograd.grad(g.float().sum(), x)


@gpu
def test_gradient_against_differences():
    """Central differences of the kernel's own loss along random directions |d| <= 1.  Its third
    derivative along d is w tau^2 (2 / tau)^3 at most for each of L and R: h^2 / 6 times 16 w / tau;
    the losses are off by their bound each."""
    import decode_token_sampling_gb300 as kps
    tau, h = 1.5, 0.02
    s, ids, val, r = _case(8, 3000, 12, torch.float32, "cuda", seed=11)
    for rest in (r, None):
        kw = dict(temperature=tau, rest=rest)
        _, grad = kps.distill_loss_grad(s, ids, val, **kw)
        for k in range(4):
            d = torch.rand(s.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(k)) * 2 - 1
            d.scatter_(1, ids[:, k:k + 1].long(), 1.0)
            up, down = (kps.distill_forward(s + e * h * d, ids, val, **kw)[0].double() for e in (1, -1))
            tol = sum(distill_reference(s + e * h * d, ids, val, tau, rest)[2] for e in (1, -1))
            rounding = (s.abs().max() + 1) * U * 2  # of s + h d itself, each side
            want = (grad.double() * d.double()).sum(1)
            lim = tol / (2 * h) + h * h / 6 * 16 / tau + 2 * rounding / h * tau
            assert bool(((up - down) / (2 * h) - want).abs().le(lim).all())


@gpu
def test_streams_and_graphs():
    import decode_token_sampling_gb300 as kps
    s, ids, val, r = _case(9, 20000, 32, torch.bfloat16, "cuda", seed=12)
    want_loss, want_grad = kps.distill_loss_grad(s, ids, val, rest=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        a = kps.distill_loss_grad(s, ids, val, rest=r, stream=side)
        b = kps.distill_loss_grad(s, ids, val, rest=r)  # two at once
        torch.cuda.synchronize()
        for loss, grad in (a, b):
            assert torch.equal(loss, want_loss) and torch.equal(grad, want_grad)
    graphs = []
    for _ in range(2):  # two captured calls, replayed side by side on other inputs
        x = torch.zeros_like(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = kps.distill_loss_grad(x, ids, val, rest=r)
        graphs.append((x, graph, out))
    for x, _, _ in graphs:
        x.copy_(s)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0][1].replay()
    graphs[1][1].replay()
    torch.cuda.synchronize()
    for _, _, (loss, grad) in graphs:
        assert torch.equal(loss, want_loss) and torch.equal(grad, want_grad)
    # the autograd pair captured whole (the leaf is made inside the capture) gives the eager calls' bits
    want_loss, stats = kps.distill_forward(s, ids, val, rest=r)
    want_grad = kps.distill_backward(torch.ones(9, device="cuda"), s, ids, val, stats, rest=r)
    x = s.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        leaf = x.detach().requires_grad_()
        loss = kps.distill_loss(leaf, ids, val, rest=r)
        grad, = torch.autograd.grad(loss.sum(), leaf)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want_loss) and torch.equal(grad, want_grad)


@gpu
def test_more_than_2_to_31_elements():
    """Row offsets past 32 bits: the last rows of a batch of 3.0e9 logits."""
    import decode_token_sampling_gb300 as kps
    N, V, K = 20000, 151936, 8
    s, ids, val, r = _case(6, V, K, torch.bfloat16, "cuda", seed=13)
    rows = torch.tensor([0, 1, 14133, 14134, N - 2, N - 1], device="cuda")
    big = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    big[rows] = s
    weight = torch.zeros(N, device="cuda")
    weight[rows] = 1.0
    all_ids = torch.zeros(N, K, dtype=torch.int32, device="cuda")
    all_ids[rows] = ids
    all_val = torch.zeros(N, K, device="cuda")
    all_val[rows] = val
    all_rest = torch.zeros(N, device="cuda")
    all_rest[rows] = r
    loss, grad = kps.distill_loss_grad(big, all_ids, all_val, rest=all_rest, weight=weight)
    ref_loss, ref, tol, gtol = distill_reference(s, ids, val, 1.0, r)
    half = torch.finfo(torch.bfloat16).eps / 2
    _compare(loss[rows].double(), ref_loss, tol, "loss")
    _compare(grad[rows].double(), ref, gtol + half * ref.abs() + half * gtol, "grad")
    assert float(loss.double().sum()) == pytest.approx(float(loss[rows].double().sum()))
    assert bool((grad[14000] == 0).all()) and bool((grad[N - 3] == 0).all())


@gpu
@pytest.mark.parametrize("call", ["distill_loss_grad", "distill_forward", "top_logits"])
def test_first_call_of_a_process_may_be_captured(call):
    """Nothing is set up by an earlier eager call (a process of its own)."""
    import os
    import subprocess
    import sys
    code = f"""
import torch, decode_token_sampling_gb300 as kps
s = torch.randn(3, 9000, device="cuda"); ids = torch.arange(12, device="cuda", dtype=torch.int32).view(3, 4)
val = torch.randn(3, 4, device="cuda"); args = (s, 200) if {call!r} == "top_logits" else (s, ids, val)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = kps.{call}(*args)
g.replay(); torch.cuda.synchronize()
want = kps.{call}(*args)
torch.cuda.synchronize()
assert all(a is b or torch.equal(a, b) for a, b in zip(out, want))
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@gpu
def test_two_threads_at_once():
    """Calls of different shapes from two host threads, each on a stream of its own."""
    import threading
    import decode_token_sampling_gb300 as kps
    cases = [_case(30, 20000, 32, torch.bfloat16, "cuda", seed=20), _case(7, 151936, 300, torch.float32, "cuda", seed=21)]
    want = [kps.distill_loss_grad(s, ids, val, rest=r) for s, ids, val, r in cases]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            s, ids, val, r = cases[i]
            for _ in range(20):
                got[i] = kps.distill_loss_grad(s, ids, val, rest=r, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for (loss, grad), (l, g) in zip(want, got):
        assert torch.equal(loss, l) and torch.equal(grad, g)


@gpu
def test_binding_refusals():
    import decode_token_sampling_gb300 as kps
    s, ids, val, r = _case(4, 100, 8, torch.float32, "cuda")
    for bad in (dict(student=s.half()), dict(student=s[0]), dict(student=s.t().contiguous().t()),
                dict(student=s[:1].expand(4, 100)), dict(student=s[:, ::2]), dict(ids=ids.long()), dict(ids=ids[:3]),
                dict(ids=ids[:, ::2], values=val[:, ::2]), dict(values=val.double()), dict(values=val[:, :4]),
                dict(rest=r[:2]), dict(rest=r.double()), dict(rest=r.cpu()), dict(weight=torch.ones(4)),
                dict(ids=torch.zeros(4, 1025, dtype=torch.int32, device="cuda"), values=torch.zeros(4, 1025, device="cuda"))):
        kw = dict(student=s, ids=ids, values=val)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError)):
            kps.distill_loss(**kw)
    with pytest.raises(kps.KpsError):
        kps.distill_loss(s, ids, val, temperature=0.0)
    assert kps.distill_loss(s[:0], ids[:0], val[:0]).shape == (0,)


@gpu
def test_gradient_of_rows_far_apart():
    """One row out of every 64 of a batch (the last position of each sequence): a gradient of the rows' own size."""
    import decode_token_sampling_gb300 as kps
    N, V = 6, 1003
    s, ids, val, r = _case(N, V, 12, torch.float32, "cuda", seed=9)
    buf = torch.zeros(N, 64, V, device="cuda")
    view = buf[:, -1]
    view.copy_(s)
    check(view, ids, val, 1.0, r)
    _, grad = kps.distill_loss_grad(view, ids, val, rest=r)
    assert grad.untyped_storage().nbytes() <= N * (V + 3) * 4


@gpu
@pytest.mark.parametrize("dtype,edge", [(torch.float32, 401408), (torch.bfloat16, 802816)])
@pytest.mark.parametrize("K", [960, 961, 1024])
def test_longest_lists_on_the_longest_rows_in_shared_memory(dtype, edge, K):
    """Where the row and the arrays of a long list together fill a block's shared memory."""
    for V in (edge, edge + 8, edge + 3000):
        s, ids, val, r = _case(2, V, K, dtype, "cuda", seed=K)
        check(s, ids, val, 1.0, r)


def _finite_grad(s, ids, val, tau, rest, weight=None):
    """The fused call and the pair against the formulas where the losses are huge or infinite."""
    import decode_token_sampling_gb300 as kps
    kw = dict(temperature=tau, rest=rest, weight=weight)
    want, ref, _, _ = distill_reference(s, ids, val, tau, rest, weight)
    loss, stats = kps.distill_forward(s, ids, val, **kw)
    loss2, grad = kps.distill_loss_grad(s, ids, val, **kw)
    back = kps.distill_backward(None, s, ids, val, stats, **kw)
    for got in (loss, loss2):
        # p's exponentials and their sum, and a few roundings more: all relative, the loss is no difference here
        lim = (1e-5 * want.abs()).where(torch.isfinite(want), torch.zeros_like(want))
        _compare(got.double(), want, lim, "loss")
    half = torch.finfo(s.dtype).eps / 2
    w = torch.ones_like(want) if weight is None else weight.double()
    for got in (grad, back):
        # masses below one in sums off by 1e-5
        lim = (3e-5 * (w * tau).abs())[:, None] + half * ref.abs()
        _compare(got.double(), ref, lim, "grad")


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("K", [1, 16])
def test_student_without_the_lists_tokens(dtype, tau, K):
    """-inf or the type's lowest value at every token of the teacher's list, or at one of them: a loss of
    +inf, or a huge one; next to no mass in the list: the loss of the rest alone."""
    import decode_token_sampling_gb300 as kps
    s, ids, val, r = _case(6, 3000, K, dtype, "cuda", seed=31)
    lowest = torch.finfo(dtype).min
    for value in (-math.inf, lowest, -1e9):
        x = s.clone()
        x[:3].scatter_(1, ids[:3].long(), value)
        x[3:].scatter_(1, ids[3:, :1].long(), value)
        w = torch.full((6,), 0.25 if value == lowest else 1.0, device="cuda")
        for rest in (None, r, r + 3.0, r - 3.0):
            _finite_grad(x, ids, val, tau, rest, w)
    # the lowest value everywhere but in the list: a loss of the rest's share of it, and a gradient that
    # is that share in equal parts (64 bits lose the logarithm of their number beside the lowest value)
    x = torch.full_like(s, lowest).scatter_(1, ids.long(), s.gather(1, ids.long()))
    for rest in (r, r + 3.0, r - 3.0):
        kw = dict(temperature=tau, rest=rest, weight=torch.full((6,), 0.25, device="cuda"))
        want, _, _, _ = distill_reference(x, ids, val, tau, rest, kw["weight"])
        loss, stats = kps.distill_forward(x, ids, val, **kw)
        loss2, grad = kps.distill_loss_grad(x, ids, val, **kw)
        back = kps.distill_backward(None, x, ids, val, stats, **kw)
        for got in (loss, loss2):
            _compare(got.double(), want, 1e-5 * want.abs(), "loss")
        p_rest = torch.softmax(torch.cat([val.double() / tau, rest.double()[:, None]], 1), 1)[:, -1]
        share = (-0.25 * tau * p_rest / (3000 - K))[:, None]
        for got in (grad, back):
            outside = got.double().scatter(1, ids.long(), share.expand(6, K))
            assert bool(((outside - share).abs() <= share.abs() * (1e-5 + torch.finfo(dtype).eps / 2)).all())
    # the teacher's list has no mass that fp32 holds, the student's list none at all
    x = s.clone()
    x.scatter_(1, ids.long(), -math.inf)
    far = torch.full((6,), 2000.0, device="cuda")
    loss, stats = kps.distill_forward(x, ids, val, temperature=tau, rest=far)
    loss2, grad = kps.distill_loss_grad(x, ids, val, temperature=tau, rest=far)
    assert bool((loss.abs() <= 1e-5 * tau * tau).all()) and bool((loss2.abs() <= 1e-5 * tau * tau).all())
    assert bool((grad.float().abs() <= 1e-5 * tau).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_teacher_of_the_types_lowest_values(dtype, tau):
    """A list of nothing but the lowest value is a uniform one (without a rest, or with one of -inf); with
    a rest it weighs nothing.  Largest values likewise."""
    s, ids, val, r = _case(4, 2000, 9, dtype, "cuda", seed=32)
    for vt in (torch.float32, torch.bfloat16):
        low = torch.full_like(val, torch.finfo(vt).min, dtype=vt)
        none = torch.full_like(r, -math.inf)
        none[1] = torch.finfo(torch.float32).min
        for v in (low, -low):
            check(s, ids, v, tau, None)
            check(s, ids, v, tau, torch.full_like(r, -math.inf) if v is low else none)
            check(s, ids, v, tau, r)
        # a teacher's row that is masked all over, as top_logits hands it on at temperature 1: every class alike
        check(s, ids, low, 1.0, torch.full_like(r, torch.finfo(vt).min))
        check(s, ids, -low, 1.0, torch.full_like(r, torch.finfo(vt).max))


@pytest.mark.parametrize("call", [_forward, _loss_grad, _backward])
def test_temperatures_whose_square_is_no_normal_number_are_refused(lib, call):
    """The loss holds the square of the temperature."""
    for tau in (2e-20, 1e-30, 2e19, 1e38):
        assert call(lib, tau=tau) == 1, tau
    if not torch.cuda.is_available():
        for tau in (1e-18, 1e18):
            assert call(lib, tau=tau) == 4, tau


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_rows_share_the_students_phase(dtype):
    """Every row of the gradient starts as far behind a 16-byte boundary as the student's, whatever
    the student's offset and row stride are: only then are rows stored 16 bytes at a time."""
    import decode_token_sampling_gb300 as kps
    es = torch.empty(0, dtype=dtype).element_size()
    for N, V, ld in ((1, 1000, 1000), (3, 1000, 1000), (4, 1001, 1001), (5, 1001, 1100), (2, 7, 5000)):
        for off in range(16 // es):
            student = torch.empty(off + N * ld, dtype=dtype)[off:].view(N, ld)[:, :V]
            grad = kps._grad_like(student)
            assert grad.shape == student.shape and grad.dtype == dtype and grad.stride(1) == 1
            assert grad.untyped_storage().nbytes() <= (N * (V + 16 // es) + 16 // es) * es
            for i in range(N):
                assert (grad[i].data_ptr() - student[i].data_ptr()) % 16 == 0
            if ld == V and off == 0:
                assert grad.is_contiguous()


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rest", [False, True])
def test_small_divergence_to_a_hundredth(dtype, rest):
    """A student next to its teacher, logits on a grid that makes every difference exact: the error left is
    that of the masses.  With e = 2^-22 + 2^-23 (an exponential and the roundings behind it), a share P
    of the two rests together, each a sum whose terms of exponent z are off by (2 u z + 2^-22) ln 2 and
    which adds (V / 2048 + 16) roundings, the loss is off by
    tau^2 (2 e + e' P + 16 u (1 + sum p |ln p - ln q|)) at most."""
    import decode_token_sampling_gb300 as kps
    V, K, N, tau = 4096, 64, 40, 1.0
    step = 2.0 ** (-8 if dtype == torch.float32 else -4)
    g = torch.Generator("cuda").manual_seed(33)
    t = torch.randn(N, V, device="cuda", generator=g) - (0.0 if rest else 9.0)
    t[:, :K] = 6.0 + 1.5 * torch.randn(N, K, device="cuda", generator=g)
    t = (t.clamp(-15.0, 12.0) / step).round() * step
    noise = torch.randint(-6, 7, (N, V), device="cuda", generator=g) * step
    s = (t + noise).to(dtype)
    assert torch.equal(s.float(), t + noise)
    ids = torch.arange(K, device="cuda", dtype=torch.int32).repeat(N, 1)
    val = t[:, :K].contiguous()
    r = torch.logsumexp(t[:, K:].double(), 1).float() if rest else None
    want, _, _, _ = distill_reference(s, ids, val, tau, r)
    a, b = torch.log_softmax(t.double(), 1), torch.log_softmax(s.double(), 1)
    P = a[:, K:].exp().sum(1) + b[:, K:].exp().sum(1)
    e = 2.0 ** -22 + 2.0 ** -23
    z = 40 * 1.4427  # no logit lies further below the list's largest
    e_rest = (2 * U * z + 2.0 ** -22) * 0.6932 + (V / 2048 + 16) * U
    spread = (a[:, :K].exp() * (a - b)[:, :K].abs()).sum(1)
    tol = tau * tau * (2 * e + e_rest * P + 16 * U * (1 + spread))
    assert bool((tol <= want / 10).all())  # a bound that a wrong loss would not meet
    kw = dict(temperature=tau, rest=r)
    for got in (kps.distill_forward(s, ids, val, **kw)[0], kps.distill_loss_grad(s, ids, val, **kw)[0]):
        _compare(got.double(), want, tol, "loss")


def test_misaligned_results_and_statistics_are_refused(lib):
    """Addresses that the kernels would read or write as floats."""
    off = ctypes.c_void_p((1 << 28) + 2)
    assert _forward(lib, loss=off) == 1
    assert _forward(lib, stats=off) == 1
    assert _loss_grad(lib, loss=off) == 1
    assert _backward(lib, stats=off) == 1
    assert _backward(lib, grad_loss=off) == 1


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tau", [0.0625, 1.0, 16.0])
def test_teacher_with_a_rest_far_from_zero(dtype, tau):
    """Logits whose quotients by the temperature lie far from zero: the rest, a float of that size, and the
    list's classes differ by a few nats all the same."""
    import decode_token_sampling_gb300 as kps
    s, _, _, _ = _case(6, 3000, 8, torch.float32, "cuda", seed=34)
    g = torch.Generator("cuda").manual_seed(35)
    t = (s + torch.randn(s.shape, device="cuda", generator=g)) * tau
    for shift in (-1e3, 3e4, -3e4, 1e6, -1e9):
        x = (s * tau + shift).to(dtype)
        top = kps.top_logits((t + shift).contiguous(), 8, temperature=tau)
        for nudge in (0.0, 3.0, -3.0):
            check(x, top.ids, top.values, tau, top.rest + nudge)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [-3e4, -500.0, 500.0, 3e4])
def test_gradient_of_a_list_without_student_mass(dtype, shift):
    """-inf at every token of the list and the rest of the row far from zero: the list's gradient is minus its
    masses, whatever the loss (+inf)."""
    for K in (1, 12):
        for V in (500, 100001):
            s, ids, val, r = _case(4, V, K, torch.float32, "cuda", seed=36)
            s = (s + shift).to(dtype)
            s.scatter_(1, ids.long(), -math.inf)
            for tau in (0.25, 1.0):
                for rest in (None, r):
                    _finite_grad(s, ids, val, tau, rest)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_list_far_below_a_row_whose_largest_logit_lies_outside_the_vectors(dtype):
    """The first and last logits of rows off a 16-byte boundary are read apart from the others: neither
    they nor the others may hide how far above the list the row lies."""
    N, V = 16, 35
    g = torch.Generator("cuda").manual_seed(37)
    for top, rest_of_row in ((89.5, 86.0), (86.0, 89.5), (100.0, 87.0), (300.0, 290.0)):
        s = rest_of_row + torch.rand(N, V, device="cuda", generator=g)
        s[:, 0] = top
        s[:, 34] = top - 0.5
        s[:, 17] = 0.0
        s = s.to(dtype)
        ids = torch.full((N, 1), 17, dtype=torch.int32, device="cuda")
        val = torch.zeros(N, 1, device="cuda")
        for r in (None, torch.zeros(N, device="cuda"), torch.full((N,), 2.0, device="cuda")):
            check(s, ids, val, 1.0, r)


@gpu
@pytest.mark.parametrize("tau", [0.25, 0.5])
def test_losses_near_the_largest_number(tau):
    """fp32's lowest value at all of the teacher's mass but 2^-50: the distance is the largest number there is,
    the loss a quarter of it or less."""
    N, V, K = 64, 300, 8
    g = torch.Generator("cuda").manual_seed(38)
    s = torch.randn(N, V, device="cuda", generator=g)
    ids = torch.arange(K, device="cuda", dtype=torch.int32).repeat(N, 1)
    val = torch.randn(N, K, device="cuda", generator=g) * tau
    val[:, 7] = -35.0 * tau
    s[:, :7] = torch.finfo(torch.float32).min
    _finite_grad(s, ids, val, tau, None, torch.full((N,), 0.5, device="cuda"))
    _finite_grad(s, ids, val, tau, torch.full((N,), -35.0, device="cuda"), torch.full((N,), 0.5, device="cuda"))
