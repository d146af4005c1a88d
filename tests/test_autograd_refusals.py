"""What the differentiable operators refuse: second derivatives, forward mode, vmap.

Without a GPU the binding runs against a library that computes nothing, on CPU tensors that say they are CUDA ones: what autograd
records and what reaches the library is the binding's own.
"""

import pytest
import torch

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


gpu = pytest.mark.gpu


@gpu
def test_second_derivatives_of_logprobs_on_the_gpu():
    _second_derivatives(_logprobs, torch.randn(3, 10, device="cuda", requires_grad=True))


@gpu
def test_second_derivatives_of_the_distillation_on_the_gpu():
    _second_derivatives(_distill, torch.randn(3, 10, device="cuda", requires_grad=True))
