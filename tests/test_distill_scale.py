"""distill_loss's gradient of small weights where the logits of a row's first tokens are far below its largest: the row's sum is kept
relative to them."""
import numpy as np
import pytest
import torch

from test_distill_loss import compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [9001, 40_000, 128_256])
@pytest.mark.parametrize("T", [1.0, 0.25])
def test_small_weights_of_peaked_rows(smcsd, rest, dtype, V, T):
    """60 nats between the row's likely tokens, which stand behind every block's first vectors, and all others."""
    R, K, n = 4, 12, 40
    gen = torch.Generator("cuda").manual_seed(V)
    z = torch.randn(R, V, device="cuda", generator=gen) * 0.1 - 60 * T
    first = 8000 if V < 10_000 else 16_000 if V < 50_000 else 30_000
    z[:, first:first + n] = torch.randn(R, n, device="cuda", generator=gen) * T
    z = z.to(dtype)
    logp = torch.log_softmax(z.float() / T + torch.randn(R, V, device="cuda", generator=gen) * 0.5, 1)
    values, tokens = logp.topk(K, 1)
    weight = torch.tensor([1.0, 2.0 ** -20, 2.0 ** -50, -(2.0 ** -60)], device="cuda")
    loss, grad, status = compare(smcsd, z, tokens.int(), values.contiguous(), V, T, rest, weight)
    assert status == 0
    # unlisted likely tokens have gradients of their weight's size
    big = grad[:, first:first + n].double().abs().sum(1) / weight.double().abs()
    assert (big > 0.01).all()
    assert np.isfinite(big.cpu().numpy()).all()


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.25, 0.75, 1.0, 2.0])
def test_listed_tokens_masked_with_the_lowest_value(smcsd, rest, dtype, T):
    """The draft masks a token that the teacher gives a hundredth to: its log q may pass float32's range while its part of the loss,
    -p log q, does not."""
    R, V, K = 6, 3000, 8
    gen = torch.Generator("cuda").manual_seed(3)
    z = torch.randn(R, V, device="cuda", generator=gen).to(dtype)
    tokens = torch.rand(R, V, device="cuda", generator=gen).topk(K, 1).indices
    p = torch.full((R, K), 0.13, device="cuda")
    p[:, 5] = 0.01
    z[:3, :100] = torch.finfo(dtype).min
    z[:3] = z[:3].scatter(1, tokens[:3], 0.5).scatter(1, tokens[:3, 5:6], torch.finfo(dtype).min)
    loss, _, status = compare(smcsd, z, tokens.int(), p.log(), V, T, rest)
    assert status == 0
    assert bool(torch.isfinite(loss).all()) and bool((loss[:3] > 1e36).all()) and bool((loss[3:] < 100).all())
    alone, _, _ = compare(smcsd, z, tokens.int(), p.log(), V, T, rest, grad=False)
    assert bool(torch.isfinite(alone).all())
