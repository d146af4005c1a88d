"""The min-p stage of the sampling step (kps_sample_min_p) against its definition in 64 bits.

The reference takes the oracle's row terms before top-p (transformed row x, order, weights e,
their sum S) and applies top-p, then min-p, then the race in float64.  A row whose top-p boundary
or whose two best race scores lie within 1e-6 of each other (the sampling step's near-tie rule) is
not compared; the tests bound how many those are.
"""

import ctypes
import math

import numpy as np
import pytest

import oracle
from decode_token_sampling_gb300.workloads import f32_to_bf16_bits, make_random, make_workload

NEAR = 1e-6


def reference_row(inp, b, mp):
    """(chosen, kept indices, near tie) of one row."""
    t = oracle.row_terms(inp, b)
    x, order, e, S, nK = t["x"].astype(np.float64), t["order"], t["e"], t["S"], t["nK"]
    p, mp = float(inp.top_p[b]), float(mp)
    near = False
    c = np.cumsum(e)
    if t["greedy"] or p <= 0.0:
        n = 1
    elif p < 1.0:
        n = min(int(np.searchsorted(c, p * S, side="left")) + 1, nK)
        near = bool(np.abs(c - p * S).min() < NEAR * p * S)
    else:
        n = nK
    n_top = n
    if n > 1 and mp > 0.0:
        M = x[order[0]]
        if math.isinf(M):
            kept = x[order] == M
        else:
            with np.errstate(invalid="ignore"):
                kept = x[order] - M >= math.log(min(mp, 1.0))
        n = min(n, int(kept.sum()))
    near = near and n >= n_top - 1  # the top-p boundary decides
    ids = order[:n]
    if inp.q is None:
        return int(order[0]), ids, near
    with np.errstate(divide="ignore", invalid="ignore"):
        r = e[:n] / (inp.q[b, ids] + np.float32(inp.eps)).astype(np.float64)
    if np.isnan(r).all():
        return int(order[0]), ids, near
    r = np.where(np.isnan(r), -1.0, r)
    best = r.max()
    chosen = int(ids[r == best].min())
    others = r[ids != chosen]
    if others.size and best > 0 and not math.isinf(best):
        near = near or bool(best - others.max() < NEAR * best)
    return chosen, ids, near


def test_reference_against_brute_force():
    """On tiny rows: the kept set is every token whose probability is at least min_p of the largest."""
    inp = make_random(40, 9, seed=4, k_range=(0, 0), p_range=(1.0, 1.0))
    for b in range(40):
        mp = (0.01, 0.1, 0.5, 0.999)[b % 4]
        _, ids, _ = reference_row(inp, b, mp)
        z = inp.logits[b] / inp.temperature[b]
        pr = np.exp(z.astype(np.float64)) / np.exp(z.astype(np.float64)).sum()
        assert sorted(ids.tolist()) == np.nonzero(pr >= mp * pr.max())[0].tolist()


def test_refusals():
    from decode_token_sampling_gb300 import build
    build.build()
    import decode_token_sampling_gb300 as kps
    lib = kps.load_library()
    fake = ctypes.c_void_p(1 << 20)
    opts = kps.StepOpts(None, 0, 0, 0, None, 0, None, None, 0, 0)

    def call(**over):
        a = dict(logits=fake, dt=0, B=4, V=100, top_k=fake, top_p=fake, min_p=fake, temperature=fake, indptr=None, ids=None,
                 penalty=None, opts=ctypes.byref(opts), eps=1e-20, need=0, out_idx=fake, out=None, ws=fake, n=256, stream=None)
        a.update(over)
        return lib.kps_sample_min_p(*a.values())

    assert call(min_p=None) == 1
    assert call(min_p=ctypes.c_void_p((1 << 20) + 2)) == 1
    assert call(opts=None) == 1
    assert call(dt=9) == 1 and call(V=0) == 1 and call(top_k=None) == 1 and call(ws=None) == 3
    bad = kps.StepOpts(None, 0, 0, 0, None, 0, None, None, 0, 4)
    assert call(opts=ctypes.byref(bad)) == 1
    assert call(B=0, min_p=None) == 0
    import torch
    if not torch.cuda.is_available():
        assert call() == 4


gpu = pytest.mark.gpu
POLICIES = (0, 1, 2, 3)


def run(inp, min_p, kernel, need_logits=True, **kw):
    import torch
    import decode_token_sampling_gb300 as kps
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    logits = d(inp.logits.view(np.int16)).view(torch.bfloat16) if inp.dtype == "bf16" else d(inp.logits)
    if inp.seen_indptr is not None:
        kw.update(seen_indptr=d(inp.seen_indptr), seen_ids=d(inp.seen_ids), penalty=d(inp.penalty))
    idx, filt = kps.sample(logits, d(inp.top_k), d(inp.top_p), d(inp.temperature), None if inp.q is None or "seed" in kw else d(inp.q),
                           eps=inp.eps, min_p=None if min_p is None else d(min_p), need_logits=need_logits, kernel=kernel, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), None if filt is None else filt.cpu().numpy()


def check(inp, min_p, kernel, most_near=0.1, **kw):
    min_p = np.asarray(min_p, np.float32)
    want = [reference_row(inp, b, min_p[b]) for b in range(inp.B)]
    for need in (True, False):
        idx, filt = run(inp, min_p, kernel, need, **kw)
        bad = []
        for b, (chosen, ids, near) in enumerate(want):
            if near:
                continue
            if idx[b] != chosen:
                bad.append((b, "chosen", int(idx[b]), chosen))
            if need:
                x = oracle.row_terms(inp, b)["x"]
                row = np.full(inp.V, -np.inf, np.float32)
                row[ids] = x[ids]
                if not np.array_equal(filt[b], row):
                    bad.append((b, "filtered", int((filt[b] != -np.inf).sum()), len(ids)))
        assert not bad, f"{len(bad)} of {inp.B}: {bad[:8]}"
    assert sum(w[2] for w in want) <= max(1, most_near * inp.B)


def mixed(B, seed=0):
    r = np.random.default_rng(seed)
    m = r.uniform(0.01, 0.4, B).astype(np.float32)
    odd = np.array([0.0, np.nan, -1.0, 1.0, 2.0, 1e-30, 0.999, 1e-4, np.inf], np.float32)
    at = np.arange(B) % 4 == 3
    m[at] = odd[np.arange(at.sum()) % odd.size]
    return m


@gpu
@pytest.mark.parametrize("kernel", POLICIES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,V", [(1, 1), (5, 7), (6, 1001), (9, 4096), (9, 4099), (3, 32000), (70, 8192), (160, 20480), (2, 50001)])
def test_sizes(B, V, dtype, kernel):
    for seed, kw in ((1, {}), (2, dict(k_range=(0, 0))), (3, dict(k_range=(0, 0), p_range=(1.0, 1.0)))):
        check(make_random(B, V, seed=seed, dtype=dtype, **kw), mixed(B, seed), kernel)


@gpu
@pytest.mark.parametrize("kernel", POLICIES)
@pytest.mark.parametrize("V", [5003, 16384])
def test_ties_specials_and_penalty(V, kernel):
    for seed, kw in ((5, dict(ties=True)), (6, dict(special=True)), (7, dict(penalty=1.3, n_seen=200)),
                     (8, dict(special=True, penalty=0.8, n_seen=50, k_range=(0, 0))),
                     (9, dict(ties=True, k_range=(0, 0), p_range=(1.0, 1.0)))):
        check(make_random(66, V, seed=seed, **kw), mixed(66, seed), kernel, most_near=0.5)


@gpu
@pytest.mark.parametrize("kernel", POLICIES)
@pytest.mark.parametrize("V", [30011, 30000])
def test_rows_that_a_sample_misjudges(V, kernel):
    """Rows that overflow the list (flat, constant, a plateau), hardly any finite token, infinities,
    thousands of survivors under top-p, a maximum the sample does not see."""
    B = 72
    inp = make_random(B, V, seed=10, k_range=(0, 0))
    r = np.random.default_rng(11)
    x = inp.logits
    mp = np.full(B, 0.05, np.float32)
    x[0] = 0.25
    x[1] = r.normal(0, 0.3, V)
    x[2] = r.normal(0, 0.3, V)
    x[3] = -np.inf
    x[4] = -np.inf
    x[4, r.integers(0, V, 20)] = r.normal(0, 1, 20)
    x[5, 17] = np.inf
    x[6, r.integers(0, V, 3000)] = 9.0
    x[7, r.integers(0, V, 20)] = np.nan
    x[8] = np.nan
    x[9] = np.finfo(np.float32).min
    x[9, 100:130] = r.normal(0, 1, 30)
    x[10] = -1e4
    x[10, 7] = 5.0
    x[11, 4321] = 80.0
    for b in range(12, 30):  # about 1500 to 5000 survivors
        x[b] = r.normal(0, 1.0, V)
        inp.temperature[b] = 1.0
        mp[b] = 0.02 + 0.005 * (b - 12)
    inp.top_p[::2] = 1.0
    inp.top_p[1:30:4] = 0.3
    check(inp, mp, kernel)


@gpu
@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("V,dtype", [(262144, "bf16"), (300001, "bf16"), (262144, "f32")])
def test_largest_rows(V, dtype, kernel):
    """The row kernel's largest vocabulary, and one past it (the cluster kernel)."""
    for seed, kw in ((20, dict(k_range=(0, 0))), (21, dict(k_range=(0, 0), p_range=(1.0, 1.0)))):
        check(make_random(3, V, seed=seed, dtype=dtype, **kw), [0.02, 0.1, 0.5], kernel, most_near=0.4)


@gpu
@pytest.mark.parametrize("T", [1e-4, 1e-30, 1e30, 3e38])
def test_extreme_temperatures(T):
    """Quotients that overflow, meet or fall below the normal numbers."""
    for kernel in POLICIES:
        inp = make_random(64, 4096, seed=22, k_range=(0, 0), p_range=(1.0, 1.0))
        inp.temperature[:] = T
        inp.top_p[::2] = 0.9
        check(inp, mixed(64, 22), kernel, most_near=1.0)


@gpu
@pytest.mark.parametrize("kernel", POLICIES)
def test_border_values(kernel):
    """Elements on both sides of the border by one unit in the last place, for borders that are
    floats exactly (min_p a power of two is not: ln 2 is irrational, so the nearest floats differ)."""
    B, V = 64, 5000
    inp = make_random(B, V, seed=12, k_range=(0, 0), p_range=(1.0, 1.0), t_range=(1.0, 1.0))
    r = np.random.default_rng(13)
    mp = r.uniform(0.001, 0.9, B).astype(np.float32)
    for b in range(B):
        M = np.float32(r.uniform(5, 30)) * (1 if b % 2 else -1)
        x = inp.logits[b]
        x[:] = M - np.float32(20.0)
        x[50] = M
        edge = np.float32(np.float64(M) + math.log(np.float64(mp[b])))
        for k in range(-6, 7):
            v = edge
            for _ in range(abs(k)):
                v = np.nextafter(v, np.float32(np.inf if k > 0 else -np.inf), dtype=np.float32)
            x[100 + 37 * (k + 6)] = v
    check(inp, mp, kernel)


@gpu
@pytest.mark.parametrize("kernel", POLICIES)
def test_draw_sources_and_off_values(kernel):
    inp = make_random(68, 8192, seed=14, k_skip_frac=0.5)
    mp = mixed(68, 14)
    inp.q = None  # sampling off
    check(inp, mp, kernel)
    inp.q = oracle.exp_draws(68, 8192, 99, 3)
    check(inp, mp, kernel, seed=99, step=3)
    # min-p off in every row: what kps_sample_step gives
    off = np.tile(np.array([0.0, -1.0, np.nan, -np.inf], np.float32), 17)
    a, b = run(inp, off, kernel), run(inp, None, kernel)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("name", ["small_mixed", "bf16_zipf", "batch256_penalty", "flat_nucleus", "single_row_long"])
def test_named_workloads(name):
    rows = None if name in ("small_mixed", "single_row_long") else range(64, 64 + 64)
    if name == "bf16_zipf":
        rows = range(64)
    inp = make_workload(name, rows=rows)
    B = inp.B
    inp.top_k[::3] = 0
    inp.top_p[::6] = 1.0
    check(inp, np.random.default_rng(15).uniform(0.02, 0.2, B).astype(np.float32), 0)


@gpu
def test_step_options_with_min_p():
    """Seen bits extended in place, the end-of-sequence epilogue and generated draws over three steps."""
    import torch
    import decode_token_sampling_gb300 as kps
    B, V, eos = 66, 4100, 3
    inp = make_random(B, V, seed=16, k_range=(0, 0), p_range=(0.9, 1.0))
    mp = np.random.default_rng(17).uniform(0.05, 0.5, B).astype(np.float32)
    inp.penalty = np.full(B, 1.4, np.float32)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    bits = np.zeros((B, (V + 31) // 32), np.uint32)
    dbits = d(bits.view(np.int32))
    fin, dfin = np.zeros(B, np.uint8), torch.zeros(B, dtype=torch.uint8, device="cuda")
    unf = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, k, p, t, m, pen = (d(a) for a in (inp.logits, inp.top_k, inp.top_p, inp.temperature, mp, inp.penalty))
    for step in range(3):
        idx, _ = kps.sample(x, k, p, t, None, seed=5, step=step, penalty=pen, seen_bits=dbits, update_seen=True, finished=dfin,
                            eos_id=eos, unfinished=unf, min_p=m)
        torch.cuda.synchronize()
        inp.seen_indptr, inp.seen_ids = oracle.seen_ids_from_bits(bits, V)
        inp.q = oracle.exp_draws(B, V, 5, step)
        want = np.array([reference_row(inp, b, mp[b])[0] for b in range(B)], np.int64)
        left = oracle.eos_epilogue(want, fin, eos)
        oracle.seen_append(bits, want, V)
        assert np.array_equal(idx.cpu().numpy(), want)
        assert np.array_equal(dfin.cpu().numpy(), fin) and int(unf.item()) == left
        assert np.array_equal(dbits.cpu().numpy().view(np.uint32), bits)


@gpu
def test_binding_refusals():
    import torch
    import decode_token_sampling_gb300 as kps
    B, V = 4, 100
    one = lambda dt, v: torch.full((B,), v, dtype=dt, device="cuda")  # noqa: E731
    x = torch.randn(B, V, device="cuda")
    for bad in (one(torch.float64, 0.1), one(torch.float32, 0.1)[:3], one(torch.float32, 0.1).cpu()):
        with pytest.raises((TypeError, ValueError)):
            kps.sample(x, one(torch.int32, 0), one(torch.float32, 1.0), one(torch.float32, 1.0), None, min_p=bad)


@gpu
def test_graph_replay():
    import torch
    import decode_token_sampling_gb300 as kps
    inp = make_random(70, 8192, seed=18, k_skip_frac=0.5)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    args = [d(a) for a in (inp.logits, inp.top_k, inp.top_p, inp.temperature, inp.q)]
    mp = d(mixed(70, 18))
    ws = kps.new_workspace(70, 8192)
    out = torch.empty(70, dtype=torch.int64, device="cuda")
    want, _ = kps.sample(*args, min_p=mp, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kps.sample(*args, min_p=mp, workspace=ws, out_idx=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("penalty", [None, 1.2])
def test_top_p_border_repeats_to_the_bit(dtype, penalty):
    """Rows alike but for top_p, whose values are the floats around the share of a prefix: the target is one
    sum of fixed-point masses, so every call keeps the same set, and so does the selection over the
    whole row (KERNEL_ROW_EXACT)."""
    import torch
    import decode_token_sampling_gb300 as kps
    B, V = 96, 32768
    for seed in range(6):
        inp = make_random(B, V, seed=40 + seed, dtype=dtype, scale=3.0, k_range=(0, 0), penalty=penalty, n_seen=300)
        inp.top_k[:] = 0
        inp.logits[:] = inp.logits[0]
        inp.temperature[:] = inp.temperature[0]
        if penalty is not None:
            inp.seen_ids = np.tile(inp.seen_ids[:300], B)
        inp.top_p[:] = 0.9
        t = oracle.row_terms(inp, 0)
        e = t["e"]
        n = int((e >= 0.02).sum())
        # from half a unit in the last place to 2^-13 away on both sides, of a border inside the list and of its end
        p = np.cumsum(e)[n // 2 if seed % 2 else n - 1] / t["S"]
        away = np.arange(B) - B / 2 + 0.5
        inp.top_p[:] = p * (1 + np.sign(away) * 2.0 ** (-25 + 12 * np.abs(away) / (B / 2)))
        mp = np.full(B, 0.02, np.float32)
        runs = [run(inp, mp, kernel) for kernel in (kps.KERNEL_ROW_EXACT, kps.KERNEL_ROW, kps.KERNEL_ROW, kps.KERNEL_ROW, kps.KERNEL_AUTO)]
        for idx, filt in runs[1:]:
            assert np.array_equal(idx, runs[0][0]) and np.array_equal(filt, runs[0][1])
        kept = (runs[0][1] > -np.inf).sum(1)
        border = n // 2 + 1 if seed % 2 else n  # tokens up to the border's
        assert kept.min() == border and kept.max() == (border + 1 if seed % 2 else n)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_whose_mass_has_no_estimate(dtype):
    """Rows that rise by steps, hold NaN, a mask's value almost everywhere, magnitudes whose quotients
    lose their digits, or an extreme temperature: the kept set is the exact selection's all the same."""
    import decode_token_sampling_gb300 as kps
    B, V = 80, 24576
    inp = make_random(B, V, seed=60, dtype="f32", scale=2.0, k_range=(0, 0), p_range=(0.3, 0.99))
    inp.top_k[:] = 0
    r = np.random.default_rng(61)
    x = inp.logits
    low = -3.3895314e38
    for b in range(B):
        kind = b % 10
        if kind == 0:
            x[b] += np.floor(np.arange(V) / V * 6) * (20.0 + b)  # each step past the last one's unit
        elif kind == 1:
            x[b, r.integers(0, V, 5)] = np.nan
        elif kind in (2, 3, 4):
            keep = r.integers(0, V, 50)
            kept = x[b, keep].copy()
            x[b] = (-np.inf, -1e4, low)[kind - 2]
            x[b, keep] = kept
        elif kind == 5:
            x[b] += (1e3, -1e4, 1e5, -3e5)[b // 10 % 4]
        elif kind == 6:
            inp.temperature[b] = (1e-30, 1e-20, 1e20, 1e31)[b // 10 % 4]
        elif kind == 7:
            x[b] = low
            x[b, :3] = (5.0, 4.5, 4.0)
        elif kind == 8:
            x[b] = 0.001 * x[b]  # thousands of survivors
        else:
            x[b, : V // 2] -= 90.0
    if dtype == "bf16":
        inp.logits, inp.dtype = f32_to_bf16_bits(x), "bf16"
    mp = r.uniform(0.01, 0.3, B).astype(np.float32)
    mp[8::10] = 0.98
    runs = [run(inp, mp, kernel) for kernel in (kps.KERNEL_ROW_EXACT, kps.KERNEL_ROW, kps.KERNEL_ROW)]
    for idx, filt in runs[1:]:
        assert np.array_equal(idx, runs[0][0]) and np.array_equal(filt, runs[0][1])
    check(inp, mp, kps.KERNEL_ROW, most_near=0.3)
