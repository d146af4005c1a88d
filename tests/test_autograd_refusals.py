"""What the differentiable operators refuse: second derivatives, forward mode, vmap.

Without a GPU the binding runs against a library that computes nothing, on CPU tensors that say they are CUDA ones: what autograd
records and what reaches the library is the binding's own.
"""

import pytest
import torch
from torch.autograd import forward_ad

import decode_token_sampling_gb300 as kps


class _Library:
    """Takes every call and counts it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("kps_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(kps, "load_library", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True), raising=False)
    return lib


def _logprobs(x):
    t = kps.token_logprobs(x, torch.zeros(x.shape[0], dtype=torch.int64, device=x.device))
    return t.logprob.sum() + t.entropy.sum()


def _second_derivatives(call, x):
    """The gradient alone is given; what would go on through it raises, beside a term that has a second derivative too."""
    u, = torch.autograd.grad(call(x), x, create_graph=True)
    assert u.shape == x.shape
    with torch.no_grad():
        u.mul_(2.0)  # (a tensor of its own)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (u.pow(2).sum() + (x ** 2).sum()).backward()
    assert x.grad is None
    # with respect to what comes from above, too
    w = torch.ones((), device=x.device, requires_grad=True)
    u, = torch.autograd.grad(call(x) * w, x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(u.sum() + w * w, w)
    # and not where nothing is asked of it
    y, = torch.autograd.grad(call(x) + (x ** 2).sum(), x)
    assert not y.requires_grad


def test_second_derivatives_of_logprobs(library):
    _second_derivatives(_logprobs, torch.randn(3, 10, requires_grad=True))
    assert library.calls.count("kps_token_logprobs_backward") == 3


def _distill(x):
    n = x.shape[0]
    ids = torch.arange(3 * n, dtype=torch.int32, device=x.device).view(n, 3)
    return kps.distill_loss(x, ids, torch.zeros(n, 3, device=x.device)).sum()


def test_second_derivatives_of_the_distillation(library):
    _second_derivatives(_distill, torch.randn(3, 10, requires_grad=True))
    assert library.calls.count("kps_distill_backward") == 3


def _calls(device):
    """(call, its arguments that may carry a tangent) for every operator that says what it is not differentiated by."""
    n = 3
    g = torch.Generator().manual_seed(0)
    x = torch.randn(n, 10, generator=g).to(device)
    tokens = torch.zeros(n, dtype=torch.int64, device=device)
    ids = torch.arange(3, dtype=torch.int32, device=device).repeat(n, 1)
    row = torch.rand(n, generator=g).to(device) + 0.5
    return {
        "token_logprobs": (lambda x, T: kps.token_logprobs(x, tokens, temperature=T), (x, row)),
        "token_logprobs_forward": (lambda x, T: kps.token_logprobs_forward(x, tokens, temperature=T), (x, row)),
        "token_logprobs_backward": (lambda g, h, x, stats, T: kps.token_logprobs_backward(g, h, x, tokens, stats, temperature=T),
                                    (row, row, x, torch.ones(3, n, device=device), row)),
        "policy_loss_grad": (lambda x, old, A, ref, w, T: kps.policy_loss_grad(x, tokens, old, A, ref_logprob=ref, kl_coef=0.1, weight=w,
                                                                               temperature=T), (x, row, row, row, row, row)),
        "distill_loss": (lambda x, values, rest, w: kps.distill_loss(x, ids, values, rest=rest, weight=w), (x, torch.zeros(n, 3, device=device), row, row)),
    }


NAMES = ["token_logprobs", "token_logprobs_forward", "token_logprobs_backward", "policy_loss_grad", "distill_loss"]


def _forward_mode(name, device):
    """A tangent in any argument is refused before anything runs; none is needed to be refused for the others."""
    call, args = _calls(device)[name]
    call(*args)
    with forward_ad.dual_level():
        call(*args)  # (no tangent among them)
        for i in range(len(args)):
            dual = [forward_ad.make_dual(a, torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
            with pytest.raises(NotImplementedError, match="forward mode"):
                call(*dual)
        for i in range(len(args)):
            dual = [forward_ad.make_dual(a.clone().requires_grad_(), torch.ones_like(a)) if j == i else a for j, a in enumerate(args)]
            with pytest.raises((NotImplementedError, ValueError)):
                call(*dual)
    with pytest.raises(NotImplementedError, match="forward mode"):
        torch.func.jvp(lambda a: call(a, *args[1:])[0], args[:1], (torch.ones_like(args[0]),))


def _forward_over_reverse(call, x):
    """A tangent that comes from above reaches the recorded backward only."""
    with forward_ad.dual_level():
        w = forward_ad.make_dual(torch.tensor(2.0, device=x.device), torch.tensor(1.0, device=x.device))
        out = call(x) * w
        with pytest.raises(NotImplementedError, match="forward mode"):
            torch.autograd.grad(out, x)


@pytest.mark.parametrize("name", NAMES)
def test_forward_mode(name, library):
    _forward_mode(name, "cpu")
    assert len(library.calls) == 2


def test_forward_mode_from_above(library):
    _forward_over_reverse(_logprobs, torch.randn(3, 10, requires_grad=True))
    _forward_over_reverse(_distill, torch.randn(3, 10, requires_grad=True))
    assert not any("backward" in c for c in library.calls)


def _vmap(name, device):
    call, args = _calls(device)[name]
    for i in range(len(args)):
        many = [torch.stack([a, a]) if j == i else a for j, a in enumerate(args)]
        with pytest.raises(RuntimeError):
            torch.vmap(call, in_dims=tuple(0 if j == i else None for j in range(len(args))))(*many)


@pytest.mark.parametrize("name", NAMES)
def test_vmap(name, library):
    _vmap(name, "cpu")
    assert library.calls == []


gpu = pytest.mark.gpu


@gpu
def test_second_derivatives_of_logprobs_on_the_gpu():
    _second_derivatives(_logprobs, torch.randn(3, 10, device="cuda", requires_grad=True))


@gpu
def test_second_derivatives_of_the_distillation_on_the_gpu():
    _second_derivatives(_distill, torch.randn(3, 10, device="cuda", requires_grad=True))


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_forward_mode_and_vmap_on_the_gpu(name):
    _forward_mode(name, "cuda")
    _vmap(name, "cuda")


@gpu
def test_forward_mode_from_above_on_the_gpu():
    _forward_over_reverse(_logprobs, torch.randn(3, 10, device="cuda", requires_grad=True))
    _forward_over_reverse(_distill, torch.randn(3, 10, device="cuda", requires_grad=True))
