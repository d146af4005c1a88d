"""Tensors that a saved-tensor hook gives back to the recorded backward of token_logprobs: what is not as it was saved is
refused by name, before anything is launched; what lies elsewhere in memory is read there.

Without a GPU the binding runs against a library that records its calls, on CPU tensors that say they are CUDA ones.
"""

import pytest
import torch

import decode_token_sampling_gb300 as kps


class _Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("kps_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, args))
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


SAVED = ["logits", "tokens", "stats", "temperatures"]  # in the order in which they are saved


def _apart(t):
    """The same values with stride 2 along the last dimension."""
    return torch.stack([t, t], -1)[..., 0]


CHANGES = {
    "half": lambda t: t.half() if t.is_floating_point() else t.short(),
    "double": lambda t: t.double() if t.is_floating_point() else t.int(),
    "one row less": lambda t: t[..., :-1, :].contiguous() if t.dim() == 2 else t[:-1].contiguous(),
    "one column less": lambda t: t[..., :-1].contiguous(),
    "strides": _apart,
    "flat": lambda t: t.reshape(-1)[:1],
    "on another device": lambda t: t.to("meta"),
}


def _recorded(device, change, which, monkeypatch=None):
    """The gradient of a recorded call whose saved tensor number `which` comes back changed."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 10, generator=g).to(device).requires_grad_()
    tokens = torch.zeros(4, dtype=torch.int64, device=device)
    T = torch.ones(4, device=device)
    count = iter(range(100))
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (next(count), t), lambda it: change(it[1]) if it[0] == which else it[1]):
        t = kps.token_logprobs(x, tokens, temperature=T)
    return torch.autograd.grad(t.logprob.sum(), x)[0]


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("which", range(4), ids=SAVED)
def test_changed_tensors_never_reach_the_library(which, change, library):
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        _recorded("cpu", CHANGES[change], which)
    assert [name for name, _ in library.calls] == ["kps_token_logprobs"]


def test_logits_in_host_memory_never_reach_it(library, monkeypatch):
    """Wherever they say that they lie: a device index alone is no CUDA device."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: not self.__dict__.get("host")), raising=False)

    def host(t):
        t = t.clone()
        t.host = True
        return t

    x = torch.randn(4, 10).requires_grad_()
    t = kps.token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    ctx = t.logprob.grad_fn
    saved = ctx.saved_tensors

    class Context:
        saved_tensors = (host(saved[0].detach()), *saved[1:])
        dtype, shape, temperature = ctx.dtype, ctx.shape, ctx.temperature

    with pytest.raises(ValueError, match="CUDA"):
        kps._token_logprobs_grad(Context, torch.ones(4), None)
    assert [name for name, _ in library.calls] == ["kps_token_logprobs"]


def test_tensors_as_they_were_saved_reach_it(library):
    _recorded("cpu", lambda t: t, 0)
    _recorded("cpu", lambda t: t.clone(), 0)
    _recorded("cpu", lambda t: torch.cat([t, t], 1)[:, :10], 0)  # rows apart
    _recorded("cpu", lambda t: t.clone(), 2)
    assert [name for name, _ in library.calls] == ["kps_token_logprobs", "kps_token_logprobs_backward"] * 4
    assert [args[4] for name, args in library.calls if "backward" in name] == [10, 10, 20, 10]


gpu = pytest.mark.gpu


@gpu
def test_changed_tensors_are_refused_on_the_gpu():
    for which in range(4):
        for change in ("half", "double", "one row less", "one column less", "strides", "flat"):
            with pytest.raises((TypeError, ValueError, RuntimeError)):
                _recorded("cuda", CHANGES[change], which)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            _recorded("cuda", lambda t: t.cpu(), which)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tensors_kept_elsewhere(dtype):
    """The gradient is the same to the bit after the saved tensors have been in host memory and come back at other
    addresses, rows apart among them."""
    g = torch.Generator("cuda").manual_seed(2)
    buf = torch.randn(5, 3007, device="cuda", generator=g).to(dtype)
    x = buf[:, 1:3002].detach().requires_grad_()
    tokens = torch.tensor([0, 3000, -1, 7, 1234], device="cuda")
    T = torch.rand(5, device="cuda", generator=g) + 0.5
    u, v = torch.randn(5, device="cuda", generator=g), torch.randn(5, device="cuda", generator=g)

    def grad():
        t = kps.token_logprobs(x, tokens, 3, temperature=T)
        return lambda: torch.autograd.grad([t.logprob, t.entropy], x, [u, v])[0]

    want = grad()()
    with torch.autograd.graph.save_on_cpu():
        later = grad()
        got = later()
    assert torch.equal(got, want)
    wider = lambda t: torch.cat([t, t], 1)[:, :t.shape[1]] if t.dim() == 2 and t.shape[0] == 5 else t.clone()  # noqa: E731
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, wider):
        got = grad()()
    assert torch.equal(got, want)
