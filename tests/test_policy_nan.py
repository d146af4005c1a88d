"""NaN among what the policy loss takes beside the logits: it reaches the loss and the gradient of its row, and no other."""

import math

import pytest
import torch

gpu = pytest.mark.gpu
NAN = math.nan


def _rows(dtype, V):
    """Ten rows of one size, each but the first, the seventh and the last two with a NaN; which of them are NaN, and which 0."""
    import decode_token_sampling_gb300 as kps
    g = torch.Generator("cuda").manual_seed(V)
    x = torch.randn(10, V, device="cuda", generator=g).to(dtype)
    tokens = torch.randint(0, V, (10,), device="cuda", generator=g)
    lp = kps.token_logprobs(x, tokens).logprob
    #       plain A = NaN on both sides of the clip, inside   A = 0 with old = NaN, +inf ratio   old = NaN  weight 0, A = NaN   plain
    A = [1.0, NAN, NAN, NAN, 0.0, 0.0, -1.0, NAN, NAN, 1.0]
    step = torch.tensor([0.1, -0.5, 0.0, 0.5, 0.0, 200.0, 0.0, 0.1, -0.5, 0.1], device="cuda")
    old = lp - step
    old[4] = old[6] = NAN
    weight = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.0, 2.0, 1.0], device="cuda")
    nan = torch.tensor([0, 1, 1, 1, 1, 0, 1, 0, 1, 0], dtype=torch.bool, device="cuda")
    return x, tokens, old, torch.tensor(A, device="cuda"), weight, nan


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 5003, 1 << 20])  # in shared memory, and (the longest, fp32 and bf16) in two launches
@pytest.mark.parametrize("kl,ent", [(0.0, 0.0), (0.1, 0.05)])
def test_nan_reaches_its_row(V, dtype, kl, ent):
    import decode_token_sampling_gb300 as kps
    x, tokens, old, A, weight, nan = _rows(dtype, V)
    lp = kps.token_logprobs(x, tokens).logprob
    got = kps.policy_loss_grad(x, tokens, old, A, weight=weight, ref_logprob=lp + 0.2, kl_coef=kl, entropy_coef=ent)
    assert torch.equal(torch.isnan(got.loss), nan)
    assert torch.equal(torch.isnan(got.grad).all(1), nan) and torch.equal(torch.isnan(got.grad).any(1), nan)
    live = weight != 0  # the rows are distributions all the same
    assert bool(torch.isfinite(got.logprob).all()) and bool((got.entropy[live] > 0).all())
    # an advantage of 0 leaves nothing of a ratio that has left fp32
    if kl == 0:
        assert float(got.loss[5]) == 0 and bool((got.grad[5] == 0).all())
    assert float(got.loss[7]) == 0 and bool((got.grad[7] == 0).all())


@gpu
@pytest.mark.parametrize("V", [5003, 1 << 20])
def test_nan_of_the_reference_policy(V):
    import decode_token_sampling_gb300 as kps
    x, tokens, *_ = _rows(torch.float32, V)
    lp = kps.token_logprobs(x, tokens).logprob
    ref = lp.clone()
    ref[3] = NAN
    got = kps.policy_loss_grad(x, tokens, lp, torch.zeros_like(lp), ref_logprob=ref, kl_coef=0.1)
    want = torch.arange(10, device="cuda") == 3
    assert torch.equal(torch.isnan(got.loss), want) and torch.equal(torch.isnan(got.grad).all(1), want)
    assert torch.equal(torch.isnan(got.grad).any(1), want)


@gpu
@pytest.mark.parametrize("V", [50, 5003, 500001])
def test_nan_weights_and_masked_tokens(V):
    """A NaN weight is not 0: its row is read.  A token of probability 0 has a gradient of 0 whatever the loss."""
    import decode_token_sampling_gb300 as kps
    x, tokens, old, A, weight, _ = _rows(torch.float32, V)
    x[:, V // 2:] = -math.inf
    tokens %= V // 2
    lp = kps.token_logprobs(x, tokens).logprob
    A, weight = torch.ones_like(A), torch.ones_like(weight)
    weight[2] = NAN
    A[5] = NAN
    nan = torch.tensor([i in (2, 5) for i in range(10)], device="cuda")
    got = kps.policy_loss_grad(x, tokens, lp, A, weight=weight, entropy_coef=0.1)
    assert torch.equal(torch.isnan(got.loss), nan)
    assert torch.equal(torch.isnan(got.grad[:, :V // 2]).all(1), nan) and torch.equal(torch.isnan(got.grad).any(1), nan)
    assert bool((got.grad[:, V // 2:] == 0).all())
