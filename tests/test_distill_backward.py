"""distill_loss beside torch's autograd: the loss has no graph, the gradient goes on by logits.backward."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rest", [False, True])
def test_the_gradient_goes_on_by_backward(smcsd, rest):
    R, V, K, width = 40, 700, 12, 32
    gen = torch.Generator("cuda").manual_seed(0)
    hidden = torch.randn(R, width, device="cuda", generator=gen)
    head = (torch.randn(width, V, device="cuda", generator=gen) * 0.3).requires_grad_()
    weight = torch.rand(R, device="cuda", generator=gen)
    logits = hidden @ head
    values, tokens = torch.log_softmax(logits.detach() + torch.randn(R, V, device="cuda", generator=gen), 1).topk(K, 1)
    loss, dlogits = smcsd.distill_loss(logits, tokens.int(), values.contiguous(), V, rest=rest, weight=weight)
    assert not loss.requires_grad and not dlogits.requires_grad
    logits.backward(dlogits)
    # the formula, by autograd in float64
    head64 = head.detach().double().requires_grad_()
    logq = torch.log_softmax(hidden.double() @ head64, 1)
    p = values.double().exp() if rest else torch.softmax(values.double(), 1)
    want = (p * (p.log() - logq.gather(1, tokens))).sum(1)
    if rest:
        p_r = 1 - p.sum(1)
        q_r = logq.exp().scatter(1, tokens, 0.0).sum(1)
        want = want + p_r * (p_r.log() - q_r.log())
    (weight.double() * want).sum().backward()
    # each element of dlogits: 640 units of 2^-24 of its terms, of at most 2 a row; the product adds R of them in float32, of |hidden| < 5,
    # and the logits that the kernel saw are a float32 product of 32 terms: 40 units of 5 * 2 in the gradient's relative size
    bound = R * 5 * 2 * (640 + 40 * 10 + R) * 2.0 ** -24
    assert float((head.grad.double() - head64.grad).abs().max()) < bound
    assert float(head64.grad.abs().max()) > 100 * bound / R
    assert torch.allclose(loss.double(), want.detach(), rtol=0, atol=2e-4)
