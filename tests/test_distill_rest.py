"""distill_loss with a rest where the list leaves nothing: lists of the whole vocabulary, and of all that a grammar allows."""
import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 2), (30, 30), (250, 256), (5000, 40), (128_256, 200)])
@pytest.mark.parametrize("T", [1.0, 0.5])
def test_lists_of_all_that_has_mass(smcsd, dtype, V, K, T):
    """Draft and teacher are masked alike, and the list holds every allowed token. The sum of its probabilities is 1 but for roundings, a
    rest below 2^-21: the loss is that without a rest, to which a rest of 2^-21 adds at most 2^-21 (1 + log 2^21)."""
    R, n = 200, min(V, K)
    gen = torch.Generator("cuda").manual_seed(V)
    allowed = torch.rand(R, V, device="cuda", generator=gen).topk(n, 1).indices
    z = torch.full((R, V), ou.NEG, device="cuda").scatter(1, allowed, torch.randn(R, n, device="cuda", generator=gen) * 4).to(dtype)
    teacher = torch.log_softmax(z.float() + torch.randn(R, V, device="cuda", generator=gen), 1)
    values, tokens = teacher.gather(1, allowed), allowed.int()
    if K > n:
        values = torch.cat([values, torch.full((R, K - n), ou.NEG, device="cuda")], 1)
        tokens = torch.cat([tokens, torch.full((R, K - n), -1, device="cuda", dtype=torch.int32)], 1)
    values = values.contiguous()
    ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
    loss, grad = smcsd.distill_loss(z, tokens, values, V, temperature=T, rest=True, ws=ws)
    alone, _ = smcsd.distill_loss(z, tokens, values, V, temperature=T, rest=True, grad=False, ws=ws)
    assert smcsd.check_status(ws) == 0
    p = np.exp(host(values).astype(np.float64)).sum(1)
    assert (np.abs(1 - p) < 2.0 ** -21).all()
    want, dwant, scale, parts = ou.distill(ou.as_float64(z), host(tokens), host(values), V, T, False)
    # the values' softmax, taken again, moves their logarithms by log sum p, at most 2^-21
    for x in (loss, alone):
        assert (np.abs(ou.as_float64(x) - want) <= 128 * 2.0 ** -24 * scale + 2.0 ** -21 * (1 + 21 * np.log(2)) + 2.0 ** -21).all()
    err, half = np.abs(ou.as_float64(grad) - dwant), torch.finfo(dtype).eps / 2
    bound = (640 * 2.0 ** -24 + 2.0 ** -20) * parts
    assert (err <= bound + half * (np.abs(dwant) + bound) + 1e-30).all()
