"""Gradients at temperatures so small that an upstream gradient over the temperature leaves fp32 where the gradient does not:
rows whose largest logits are equal, or certain."""

import pytest
import torch

from token_reference import Rows, close, close_grad, policy_reference

gpu = pytest.mark.gpu
SIZES = [9, 5003, 60001]


def _rows(V, dtype):
    """Rows of steps of 1 (so that next to the largest all else is 0): one largest logit, two, four, eight equal ones, the token
    among them and not; a row of equal logits."""
    x = -(torch.arange(V, device="cuda") % 7 + 1).float().repeat(6, 1)
    for row, k in enumerate((1, 2, 4, 8, 1)):
        x[row, torch.arange(k, device="cuda") * (V // 8)] = 2.0
    x[5] = 2.0
    return x.to(dtype), torch.tensor([0, V // 8, V // 8, 0, V - 1, 3], device="cuda")


TEMPERATURES = [1.5 * 2.0 ** -127, 2.0 ** -126, 2.0 ** -120, 0.5]  # the first is no normal number: as a number for all rows only


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", SIZES)
@pytest.mark.parametrize("T", TEMPERATURES)
def test_gradients_of_logprobs(T, V, dtype):
    import decode_token_sampling_gb300 as kps
    x, tokens = _rows(V, dtype)
    one = torch.ones(6, device="cuda")
    for temperature in (T, T * one):
        if torch.is_tensor(temperature) and T < 2.0 ** -126:
            continue
        _, stats = kps.token_logprobs_forward(x, tokens, temperature=temperature)
        for g, h in ((6 * one, None), (-6 * one, 5 * one), (None, 7 * one), (0.25 * one, 0.125 * one), (1e6 * one, -1e6 * one)):
            got = kps.token_logprobs_backward(g, h, x, tokens, stats, temperature=temperature)
            want, tol = Rows(x, tokens, temperature).grad(g, h)
            close_grad(got, want, tol)
            assert not bool(torch.isnan(got).any())


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", SIZES + [1 << 20])
@pytest.mark.parametrize("T", TEMPERATURES)
def test_the_policy_loss(T, V, dtype):
    import decode_token_sampling_gb300 as kps
    x, tokens = _rows(V, dtype)
    old = kps.token_logprobs(x, tokens, temperature=T).logprob
    old = torch.where(torch.isfinite(old), old, -1.0).clamp(min=-50.0)
    A = torch.full((6,), 6.0, device="cuda")
    got = kps.policy_loss_grad(x, tokens, old, A, temperature=T, entropy_coef=3.0)
    want = policy_reference(x, tokens, old, A, ent=3.0, temperature=T)
    for name in ("logprob", "entropy", "loss"):
        close(getattr(got, name), want[name], want[name + "_tol"], name)
    close_grad(got.grad, want["grad"], want["grad_tol"])
    assert not bool(torch.isnan(got.grad).any())
