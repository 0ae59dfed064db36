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
