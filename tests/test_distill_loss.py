"""distill_loss against its formulas in float64, and its gradient against differences of the loss."""
import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

NEG = ou.NEG
# What float32 makes of it, in units of 2^-24 relative to what is added up. The loss: the exponential 4, its argument's rounding 2,
# at most 50 + 3 + 5 + 8 additions one after another and 3 scalings of 4 for the two sums, 16 for the teacher's probabilities and a few
# for the logarithms: below 128. The gradient: the same, and 4 for each unit of an exponential's argument, of which there are 126
# at most (below that it is 0): below 640.
LOSS, GRAD = 128 * 2.0 ** -24, 640 * 2.0 ** -24


def make(seed, R, V, K, dtype, std=3.0, normal=True):
    """Draft's logits, and tokens and values of a teacher that half agrees; values are log-probabilities (with `normal`)."""
    g = torch.Generator("cuda").manual_seed(seed)
    z = (torch.randn(R, V, device="cuda", generator=g) * std).to(ou.DTYPES[dtype])
    teacher = z.float() + torch.randn(R, V, device="cuda", generator=g)
    if normal:
        teacher = torch.log_softmax(teacher, 1)
    values, tokens = torch.topk(teacher, K, 1)
    return z, tokens.int(), values.contiguous()


def compare(smcsd, z, tokens, values, V, T=1.0, rest=False, weight=None, **kw):
    ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
    loss, grad = smcsd.distill_loss(z, tokens, values, V, temperature=T, rest=rest, weight=weight, ws=ws, **kw)
    status = smcsd.check_status(ws)
    want, dwant, scale, parts = ou.distill(ou.as_float64(z[:, :V]), host(tokens), host(values), V, T, rest,
                                           None if weight is None else host(weight))
    if loss is not None:
        mine = ou.as_float64(loss)
        assert np.array_equal(np.isinf(mine), np.isinf(want))
        some = np.isfinite(want)
        err = np.abs(mine[some] - want[some])
        assert (err <= LOSS * scale[some] + 1e-30).all(), np.max(err / (scale[some] + 1e-30)) * 2 ** 24
    if grad is not None:
        half = torch.finfo(z.dtype).eps / 2  # of the rounding to the gradient's type
        bound = GRAD * parts
        mine = ou.as_float64(grad)[:, :V]
        some = np.isfinite(dwant).all(1)
        err = np.abs(mine - dwant)
        ok = err <= bound + half * (np.abs(dwant) + bound) + 1e-36
        assert ok[some].all(), (np.argwhere(~ok)[:4], err[~ok][:4], dwant[~ok][:4])
    return loss, grad, status


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,V,K,T", [(1, 1, 1, 1.0), (3, 2, 1, 1.0), (2, 7, 3, 1.0), (5, 63, 8, 2.0), (4, 1000, 16, 1.0), (3, 4099, 64, 0.7), (2, 32000, 32, 2.0),
                                     (3, 32257, 256, 1.0), (2, 128256, 64, 1.0), (2, 151936, 50, 1.3), (400, 130, 5, 1.0)])
def test_sizes(smcsd, rest, dtype, R, V, K, T):
    z, tokens, values = make(V + K, R, V, K, dtype)
    weight = torch.rand(R, device="cuda") * 2 - 0.5
    assert compare(smcsd, z, tokens, values, V, T, rest, weight)[2] == 0
    assert compare(smcsd, z, tokens, values, V, T, rest, weight, grad=False)[2] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_vocabulary(smcsd, dtype):
    V = 1638368 // (2 if dtype == "bf16" else 4)
    z, tokens, values = make(1, 2, V, 20, dtype)
    assert compare(smcsd, z, tokens, values, V, rest=True)[2] == 0
    assert compare(smcsd, z, tokens, values, V, rest=True, grad=False)[2] == 0


@pytest.mark.parametrize("rest", [False, True])
def test_values_that_are_logits(smcsd, rest):
    z, tokens, values = make(5, 6, 3000, 12, "f32", normal=False)
    if not rest:  # any constant may be added to a row's values
        assert compare(smcsd, z, tokens, values + 50, 3000)[2] == 0
        assert compare(smcsd, z, tokens, values - 2000, 3000)[2] == 0
    else:  # probabilities that add up to more than one: nothing is left to the rest
        assert compare(smcsd, z, tokens, torch.log_softmax(values, 1) + 0.2, 3000, rest=True)[2] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
def test_lists_with_gaps_repeats_and_none(smcsd, dtype, rest):
    R, V, K = 9, 2500, 10
    z, tokens, values = make(7, R, V, K, dtype)
    tokens[1, 3:7] = -1
    tokens[2] = -1                      # padding: its logits may be anything
    z[2] = float("nan")
    values[2] = float("nan")
    tokens[3, 1:] = -1                  # one label
    values[3, 0] = 0.0
    tokens[4, 5] = tokens[4, 2]         # a token twice, and one in every place
    values[4] -= 1.0
    tokens[5] = tokens[5, 0].clone()
    values[5] = float(np.log(0.05))
    values[6, 4:] = NEG                 # tokens without mass
    tokens[7] = torch.arange(V - K, V, device="cuda", dtype=torch.int32)
    values[8] = NEG                     # a list without mass
    values[1, 3:7] = 1e30               # of no token
    weight = torch.linspace(0, 2, R, device="cuda")
    want, dwant = smcsd.distill_loss(z, tokens, values, V, rest=rest, weight=weight)
    assert float(want[2]) == 0 and int(dwant[2].count_nonzero()) == 0 and float(want[8]) == 0 and int(dwant[8].count_nonzero()) == 0
    assert int(dwant[0].count_nonzero()) == 0 and float(want[0]) > 0  # a weight of 0
    z[2], values[2], values[1, 3:7] = 0, 0, 0
    loss, grad, status = compare(smcsd, z, tokens, values, V, 1.0, rest, weight)
    assert status == 0 and torch.equal(loss, want) and torch.equal(grad, dwant)
    assert compare(smcsd, z, tokens, values, V, 1.0, rest, weight, grad=False)[2] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("V,K", [(300, 33), (300, 256), (20_001, 100), (128_256, 64), (128_256, 200), (151_936, 256)])
def test_long_lists_with_repeats(smcsd, dtype, rest, V, K):
    R = 6
    z, tokens, values = make(V + 3 * K, R, V, K, dtype)
    values -= 3.0                               # so that what is listed more than once leaves a rest
    tokens[1, K - 1] = tokens[1, 0]             # in the first and the last warp
    tokens[2, 1::2] = tokens[2, 0::2][: K // 2].clone()
    tokens[3, 32:] = tokens[3, : K - 32].clone()
    tokens[4] = tokens[4, 7].clone()
    tokens[5, ::3] = -1
    tokens[5, K - 1] = tokens[5, 1]
    weight = torch.linspace(0.5, 1.5, R, device="cuda")
    assert compare(smcsd, z, tokens, values, V, 1.0, rest, weight)[2] == 0
    assert compare(smcsd, z, tokens, values, V, 1.0, rest, weight, grad=False)[2] == 0


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("R,V,dtype", [(310, 21_000, "bf16"), (305, 13_001, "f32"), (80, 90_000, "bf16"), (160, 50_003, "bf16")])
def test_many_rows_in_large_shares(smcsd, rest, R, V, dtype):
    z, tokens, values = make(R + V, R, V, 40, dtype)
    weight = torch.rand(R, device="cuda") * 2 - 0.5
    assert compare(smcsd, z, tokens, values, V, 1.0, rest, weight)[2] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
def test_masked_and_far_apart_logits(smcsd, dtype, rest):
    R, V, K = 6, 3001, 8
    z, tokens, values = make(9, R, V, K, dtype)
    z[0, torch.rand(V, device="cuda") < 0.9] = NEG
    z[0].scatter_(0, tokens[0].long(), 1.0)                 # the listed ones stay
    z[1] = NEG
    z[1].scatter_(0, tokens[1].long(), torch.linspace(-1, 1, K, device="cuda").to(z.dtype))  # nothing but the list
    z[2, int(tokens[2, 0])] = NEG                           # a token that the draft forbids
    z[3] -= 300                                             # the rest is far below the list
    z[3].scatter_(0, tokens[3].long(), torch.linspace(0, 2, K, device="cuda").to(z.dtype))
    z[4].scatter_(0, tokens[4].long(), torch.full((K,), -400.0, device="cuda").to(z.dtype))  # the list far below the rest
    z[5] = torch.finfo(z.dtype).min
    z[5].scatter_(0, tokens[5].long(), torch.linspace(-1, 1, K, device="cuda").to(z.dtype))
    loss, grad, status = compare(smcsd, z, tokens, values, V, 1.0, rest)
    assert status == 0 and float(loss[2]) == float("inf")
    assert compare(smcsd, z, tokens, values, V, 1.0, rest, grad=False)[2] == 0
    if rest:  # p_r meets no mass
        assert float(loss[1]) == float("inf") and np.isfinite(float(loss[5]))  # the lowest value is a logit: log q_r = -3.4e38
        # far below, but there: its share of the gradient is the rest's own softmax
        z64 = z[3].double()
        z64[tokens[3].long()] = NEG
        p_r = 1 - values[3].double().exp().sum()
        want = -p_r * torch.softmax(z64, 0)
        free = torch.ones(V, dtype=torch.bool, device="cuda").scatter_(0, tokens[3].long(), False)
        rel = ((grad[3].double() - want).abs() / want.abs())[free]
        assert float(rel[want[free].abs() > 1e-30].max()) < 2.0 ** -8 + 1e-4


@pytest.mark.parametrize("rest", [False, True])
def test_gradient_against_differences(smcsd, rest):
    R, V, K, T, step = 4, 37, 5, 1.5, 2.0 ** -6
    z, tokens, values = make(2, R, V, K, "f32", std=1.0)
    weight = torch.tensor([1.0, 0.5, -2.0, 3.0], device="cuda")
    _, grad = smcsd.distill_loss(z, tokens, values, V, temperature=T, rest=rest, weight=weight)
    for v in range(V):
        a, b = z.clone(), z.clone()
        a[:, v] += step
        b[:, v] -= step
        la, lb = (smcsd.distill_loss(x, tokens, values, V, temperature=T, rest=rest, grad=False)[0] for x in (a, b))
        width = a[:, v].double() - b[:, v].double()
        d = (la.double() - lb.double()) / width * weight.double()
        # a central difference is off by step^2 / 6 of the third derivative, which is at most 6 / T^3; the losses by 2^-24 * 128 of about 20
        bound = weight.abs().double() * (step ** 2 / T ** 3 + 2 * LOSS * 20 / width)
        assert ((grad[:, v].double() - d).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padded_vocabularies_offsets_and_in_place(smcsd, dtype):
    R, V, K = 5, 2999, 16
    z, tokens, values = make(3, R, V, K, dtype)
    want = smcsd.distill_loss(z, tokens, values, V, rest=True)
    for start in (0, 1, 5, 8):
        wide = torch.full((R, V + 80), float("nan"), device="cuda", dtype=z.dtype)
        view = wide[:, start:]
        view[:, :V] = z
        loss, grad, status = compare(smcsd, view, tokens, values, V, rest=True)
        assert status == 0 and grad.shape == (R, V)
        assert compare(smcsd, view, tokens, values, V, rest=True, grad=False)[2] == 0
        # the same partial sums need the same places: compare with the rows' own error bounds only (in compare)
        out = torch.full((R, V + 80), 7.0, device="cuda", dtype=z.dtype)
        for at in (0, 3, 16):  # to rows that begin elsewhere
            o = out[:, at:]
            smcsd.distill_loss(view, tokens, values, V, rest=True, dlogits=o)
            assert torch.equal(o[:, :V], grad)
            assert (out[:, :at] == 7).all() and (o[:, V:] == 7).all()
            out.fill_(7.0)
        keep = wide.clone()
        loss2, grad2 = smcsd.distill_loss(view, tokens, values, V, rest=True, dlogits=view)  # in place
        assert torch.equal(loss, loss2) and torch.equal(view[:, :V], grad) and grad2.data_ptr() == view.data_ptr()
        view[:, :V] = z
        assert torch.equal(wide.isnan(), keep.isnan())
    one = z[:1].clone()
    smcsd.distill_loss(one, tokens[:1], values[:1], V, rest=True, dlogits=one)
    assert torch.equal(one, want[1][:1])


def test_either_output_alone(smcsd):
    z, tokens, values = make(4, 7, 5000, 20, "bf16")
    weight = torch.rand(7, device="cuda")
    loss, grad = smcsd.distill_loss(z, tokens, values, 5000, weight=weight)
    # the loss alone comes from another kernel, whose sums are in another order: within the bound of either
    a, none, status = compare(smcsd, z, tokens, values, 5000, weight=weight, grad=False)
    assert none is None and status == 0 and a.shape == loss.shape
    none, b = smcsd.distill_loss(z, tokens, values, 5000, weight=weight, with_loss=False)
    assert none is None and torch.equal(b, grad)
    weight[3] = 0
    z[3, 5] = float("nan")  # nothing is wanted of this row
    ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
    _, b = smcsd.distill_loss(z, tokens, values, 5000, weight=weight, with_loss=False, ws=ws)
    assert smcsd.check_status(ws) == 0 and int(b[3].count_nonzero()) == 0 and torch.equal(b[:3], grad[:3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_numbers_and_tokens_are_reported_and_the_other_rows_are_right(smcsd, dtype):
    R, V, K = 4, 40_001, 6
    z, tokens, values = make(6, R, V, K, dtype)
    want, dwant = smcsd.distill_loss(z, tokens, values, V, rest=True)
    walone, _ = smcsd.distill_loss(z, tokens, values, V, rest=True, grad=False)
    others = [0, 1, 3]

    def check(code, z=z, tokens=tokens, values=values, rows=others):
        ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
        loss, grad = smcsd.distill_loss(z, tokens, values, V, rest=True, ws=ws)
        assert smcsd.check_status(ws) == code
        assert torch.equal(loss[rows], want[rows]) and torch.equal(grad[rows], dwant[rows])
        assert smcsd.check_status(ws) == 0
        alone, _ = smcsd.distill_loss(z, tokens, values, V, rest=True, grad=False, ws=ws)
        assert smcsd.check_status(ws) == code and torch.equal(alone[rows], walone[rows])
    for where in (0, 20_000, V - 1, int(tokens[2, 0])):
        for bad in (float("nan"), float("inf")):
            x = z.clone()
            x[2, where] = bad
            check(smcsd.ERR_NONFINITE, z=x)
    x = z.clone()
    x[2] = NEG
    check(smcsd.ERR_NONFINITE, z=x)
    for bad in (float("nan"), float("inf")):
        v = values.clone()
        v[2, 3] = bad
        check(smcsd.ERR_NONFINITE, values=v)
    for bad in (V, -2, 2 ** 31 - 1, -2 ** 31):
        t = tokens.clone()
        t[2, 4] = bad
        check(smcsd.ERR_RANGE, tokens=t)


def test_a_call_repeats_its_bits_and_runs_captured(smcsd):
    R, V, K = 64, 32000, 32
    z, tokens, values = make(8, R, V, K, "bf16")
    ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)
    loss, grad = torch.empty(R, device="cuda"), torch.empty_like(z)

    def call():
        smcsd.distill_loss(z, tokens, values, V, rest=True, loss=loss, dlogits=grad, ws=ws)
    want = smcsd.distill_loss(z, tokens, values, V, rest=True)
    for _ in range(5):
        call()
        assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    z2, t2, v2 = make(9, R, V, K, "bf16")
    z.copy_(z2), tokens.copy_(t2), values.copy_(v2)
    want = smcsd.distill_loss(z, tokens, values, V, rest=True)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1])


def test_a_teachers_list_from_its_logits(smcsd):
    # the target's top log-probabilities by beam_select, and the draft's loss against them; a teacher that is the draft costs nothing
    R, V, K = 32, 5003, 24
    z, _, _ = make(10, R, V, 1, "f32")
    top = smcsd.beam_select(z, R, 1, V, K, temperature=2.0)
    tokens, values = top["tokens"].view(R, K), top["scores"].view(R, K)
    for rest in (False, True):
        loss, grad, status = compare(smcsd, z, tokens, values, V, 2.0, rest)
        assert status == 0
    assert float(loss.abs().max()) < 1e-4 and float(grad.abs().max()) < 1e-5


def test_gradient_between_the_logits_rows(smcsd):
    R, V = 5, 1003
    z, tokens, values = make(11, R, V, 12, "bf16")
    want = smcsd.distill_loss(z, tokens, values, V)
    both = torch.zeros(R, 2 * V + 5, device="cuda", dtype=z.dtype)
    both[:, :V] = z
    loss, grad = smcsd.distill_loss(both[:, :V], tokens, values, V, dlogits=both[:, V:2 * V])
    assert torch.equal(loss, want[0]) and torch.equal(grad, want[1]) and torch.equal(both[:, :V], z) and int(both[:, 2 * V:].count_nonzero()) == 0
    with pytest.raises(smcsd.SMCSDError):
        smcsd.distill_loss(both[:, :V], tokens, values, V, dlogits=both[:, V - 1:2 * V - 1])
    with pytest.raises(smcsd.SMCSDError):
        smcsd.distill_loss(z, tokens, values, V, weight=loss, loss=loss)


@pytest.mark.parametrize("V", [24_000, 128_256])
def test_lists_that_change_meanwhile_harm_nobody(smcsd, V):
    """A row's blocks may read different lists where another stream writes them: the results are anything, the calls after them right."""
    R, K = 300, 32
    gen = torch.Generator(device="cuda").manual_seed(V)
    logits = torch.randn(R, V, device="cuda", generator=gen, dtype=torch.bfloat16)
    listed = torch.topk(torch.log_softmax(logits.float(), 1), K, dim=1)
    tokens, values = listed.indices.int(), listed.values
    nobody, live = torch.full_like(tokens, -1), tokens.clone()
    ws = smcsd.Workspace(smcsd.OP_DISTILL_LOSS, R)
    want = smcsd.distill_loss(logits, tokens, values, V, rest=True, ws=ws)
    out = [torch.empty_like(x) for x in want]
    loss_alone = torch.empty_like(want[0])
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(other):
            for _ in range(10):
                live.copy_(nobody)
                live.copy_(tokens)
        for _ in range(3):
            smcsd.distill_loss(logits, live, values, V, rest=True, loss=out[0], dlogits=out[1], ws=ws)
            smcsd.distill_loss(logits, live, values, V, rest=True, loss=loss_alone, grad=False, ws=ws)
    torch.cuda.synchronize()
    smcsd.check_status(ws)  # a sum from blocks that read different lists may be reported; this clears it
    smcsd.distill_loss(logits, live, values, V, rest=True, loss=out[0], dlogits=out[1], ws=ws)
    assert smcsd.check_status(ws) == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
