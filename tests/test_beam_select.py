"""beam_select against its definition in float64: sizes, ties, beams that are next to one another, finished and dead beams, masks."""
import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

NEG = ou.NEG


def make(seed, G, N, V, dtype, std=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(G * N, V, device="cuda", generator=g) * std).to(ou.DTYPES[dtype])


def compare(smcsd, logits, G, N, V, M, scores=None, finished=None, sure=1e-10, **kw):
    """Tokens, ancestors and flags equal, scores within the error of one sum (1.9e-6, see the kernel's bound; exact logits times c) and
    half a step of float32, 2^-24 of the score."""
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    got = smcsd.beam_select(logits, G, N, V, M, scores=None if scores is None else dev(scores), finished=None if finished is None else dev(finished),
                            ws=ws, **kw)
    status = smcsd.check_status(ws)
    names = dict(pad_token="pad", eos_token="eos", temperature="temperature")
    z = ou.as_float64(logits[:, :V])
    tokens, anc, score, over, gap = ou.beam_select(z, G, N, V, M, scores=scores, finished=finished, **{names[k]: v for k, v in kw.items()})
    assert gap > sure or gap == 0, gap  # the order is certain in float64
    assert np.array_equal(host(got["tokens"]).reshape(G, M), tokens)
    assert np.array_equal(host(got["ancestors"]).reshape(G, M), anc)
    assert np.array_equal(host(got["finished"]).reshape(G, M), over)
    mine = host(got["scores"]).reshape(G, M).astype(np.float64)
    assert np.array_equal(np.isneginf(mine), np.isneginf(score))
    some = np.isfinite(score)
    assert (np.abs(mine[some] - score[some]) <= 2e-6 + 2.0 ** -24 * np.abs(score[some])).all()
    return got, status


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,N,V,M,T", [
    (1, 1, 1, 1, 1.0), (1, 1, 1, 5, 1.0), (2, 1, 7, 3, 1.0), (3, 2, 5, 12, 0.7), (1, 4, 1000, 4, 1.0), (5, 3, 1023, 9, 1.3), (2, 16, 2049, 16, 1.0),
    (3, 8, 4099, 16, 0.75), (1, 64, 5003, 64, 1.0), (2, 4, 32000, 8, 1.0), (1, 256, 300, 256, 1.0), (4, 1, 32257, 64, 1.0), (1, 16, 128256, 32, 1.0),
    (2, 1, 151936, 256, 2.0), (70, 2, 999, 3, 1.0)])
def test_sizes(smcsd, dtype, G, N, V, M, T):
    rng = np.random.default_rng(G * N + V)
    scores = rng.normal(-10, 1, G * N).astype(np.float32) if N > 1 else None
    _, status = compare(smcsd, make(V + M, G, N, V, dtype), G, N, V, M, scores=scores, temperature=T)
    assert status == 0


def test_few_and_many_groups(smcsd):
    # several blocks a group, which count themselves, and a block a group
    for G in (1025, 3000):
        assert compare(smcsd, make(G, G, 1, 130, "bf16"), G, 1, 130, 4)[1] == 0
    assert compare(smcsd, make(5, 130, 8, 9001, "bf16"), 130, 8, 9001, 8, scores=np.linspace(-3, 0, 1040).astype(np.float32))[1] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("values", [1, 2, 5])
@pytest.mark.parametrize("G,N,V,M", [(2, 1, 5000, 40), (1, 4, 3001, 16), (1, 1, 40000, 256), (3, 2, 33, 64)])
def test_ties_go_to_the_lowest_beam_and_token(smcsd, dtype, values, G, N, V, M):
    rng = np.random.default_rng(values + V)
    z = rng.integers(0, values, (G * N, V)).astype(np.float32)
    z[1:] = z[:1]  # every beam alike
    logits = torch.from_numpy(z).cuda().to(ou.DTYPES[dtype])
    assert compare(smcsd, logits, G, N, V, M)[1] == 0


def test_many_tokens_next_to_one_another(smcsd):
    # falling and rising rows, and a hundred large tokens in one run: more candidates than are ranked at a time
    V = 30000
    fall = torch.linspace(10, -10, V, device="cuda")
    run = torch.full((V,), -5.0, device="cuda")
    run[7000:9000] = torch.linspace(3, 4, 2000, device="cuda")
    logits = torch.stack([fall, fall.flip(0), run, run.flip(0)])
    for M in (1, 64, 200, 256):
        assert compare(smcsd, logits, 4, 1, V, M)[1] == 0
        assert compare(smcsd, logits, 1, 4, V, M, scores=np.array([0, -0.5, -0.25, 1.0], np.float32))[1] == 0
        assert compare(smcsd, logits.bfloat16(), 2, 2, V, M, scores=np.array([0, 0.125, 0.3, 0], np.float32))[1] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_beams_whose_scores_hardly_differ(smcsd, dtype):
    # second beams moved so that one of their tokens comes next to one of the first beam's, as near as float32 scores allow
    rng = np.random.default_rng(11)
    V, M, n = 4001, 8, 24
    logits = make(3, n, 2, V, dtype)
    z = ou.as_float64(logits)
    scores = np.zeros(2 * n, np.float32)
    lse = np.log(np.exp(z).sum(1))
    for g in range(n):
        a, b = (np.sort(z[2 * g + i] - lse[2 * g + i])[::-1] for i in range(2))
        k = int(rng.integers(0, M))
        scores[2 * g] = rng.normal(-1, 0.5)
        scores[2 * g + 1] = np.float32(float(scores[2 * g]) + a[k] - b[int(rng.integers(0, M))])
    got, status = compare(smcsd, logits, n, 2, V, M, scores=scores)
    assert status == 0
    _, _, _, _, gap = ou.beam_select(z, n, 2, V, M, scores=scores)
    assert gap < 1e-6  # the hardware exponentials alone could not have told


def test_equal_rows_that_lie_differently(smcsd):
    # rows of an odd number of bf16: alike in value, at other offsets from 16 bytes
    V, N = 20011, 6
    row = make(9, 1, 1, V, "bf16")
    logits = row.repeat(N, 1)
    scores = np.full(N, -1.5, np.float32)
    got, status = compare(smcsd, logits, 1, N, V, 32, scores=scores)
    assert status == 0
    assert np.array_equal(host(got["ancestors"])[:N], np.arange(N))


def test_finished_and_dead_beams(smcsd):
    G, N, V, M = 6, 8, 5000, 12
    rng = np.random.default_rng(2)
    logits = make(1, G, N, V, "bf16")
    scores = rng.normal(-6, 2, G * N).astype(np.float32)
    finished = (rng.random(G * N) < 0.4).astype(np.int32)
    scores[rng.random(G * N) < 0.3] = NEG
    finished[:N] = 1
    scores[N:2 * N] = NEG                       # a group without any
    scores[2 * N:3 * N], finished[2 * N:3 * N] = -2.0, 1  # finished beams with equal scores
    logits[finished.astype(bool)] = float("nan")  # rows that are not read
    logits[torch.from_numpy(np.isneginf(scores)).cuda()] = float("nan")
    eos = int(logits[-1].float().nan_to_num(-1e9).argmax())
    for M in (1, N, M, 200):
        got, status = compare(smcsd, logits, G, N, V, M, scores=scores, finished=finished, pad_token=3, eos_token=eos)
        assert status == 0
        assert np.isneginf(host(got["scores"]).reshape(G, M)[1]).all()
    # every beam of a group finished: as many candidates as beams
    assert np.isfinite(host(got["scores"]).reshape(G, M)[2]).sum() == N


def test_masked_tokens_and_rows(smcsd):
    G, N, V, M = 4, 3, 2500, 20
    logits = make(4, G, N, V, "f32")
    keep = torch.rand(G * N, V, device="cuda") < 0.004
    logits = torch.where(keep, logits, torch.full_like(logits, NEG))
    logits[0] = NEG
    logits[N:2 * N] = NEG          # a group whose rows allow nothing
    logits[2 * N:3 * N] = NEG
    logits[2 * N, V - 1] = 2.0     # a group with one token
    got, status = compare(smcsd, logits, G, N, V, M, scores=np.zeros(G * N, np.float32), pad_token=7)
    assert status == 0
    assert host(got["tokens"]).reshape(G, M)[2, 0] == V - 1 and np.isfinite(host(got["scores"]).reshape(G, M)[2]).sum() == 1
    # the type's lowest value is a token like another one
    logits = torch.full((2, 300), torch.finfo(torch.float32).min, device="cuda")
    logits[1, 5] = 0
    assert compare(smcsd, logits, 1, 2, 300, 4)[1] == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinity_are_reported_and_the_other_groups_are_right(smcsd, bad, dtype):
    G, N, V, M = 3, 2, 4099, 5
    logits = make(8, G, N, V, dtype)
    scores = np.full(G * N, -1.0, np.float32)
    want = smcsd.beam_select(logits, G, N, V, M, scores=dev(scores))
    for where in (0, 2050, V - 1):
        z = logits.clone()
        z[2, where] = bad
        ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
        got = smcsd.beam_select(z, G, N, V, M, scores=dev(scores), ws=ws)
        assert smcsd.check_status(ws) == smcsd.ERR_NONFINITE
        for k in got:
            a, b = host(got[k]).reshape(G, M), host(want[k]).reshape(G, M)
            assert np.array_equal(a[[0, 2]], b[[0, 2]])
        assert (host(got["ancestors"]).reshape(G, M)[1] == 1).all()  # the other beam's
        assert smcsd.check_status(ws) == 0
    z = logits.clone()
    z[2] = NEG
    z[2, 77] = float("nan")  # among masked tokens
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    smcsd.beam_select(z, G, N, V, M, scores=dev(scores), ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_NONFINITE
    scores[3] = bad
    smcsd.beam_select(logits, G, N, V, M, scores=dev(scores), ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_NONFINITE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_a_wider_matrix(smcsd, dtype):
    # a padded vocabulary: what lies beyond V (NaN here) is not looked at, wherever the rows begin
    G, N, V, M = 2, 4, 3001, 8
    wide = torch.full((G * N, V + 90), float("nan"), device="cuda", dtype=ou.DTYPES[dtype])
    rng = np.random.default_rng(0)
    scores = rng.normal(0, 1, G * N).astype(np.float32)
    for start in (0, 1, 7, 8, 33):
        view = wide[:, start:]
        wide.fill_(float("nan"))
        view[:, :V] = make(start, G, N, V, dtype)
        assert compare(smcsd, view, G, N, V, M, scores=scores)[1] == 0


def test_scores_far_from_zero_and_large_logits(smcsd):
    G, N, V, M = 2, 4, 3000, 16
    rng = np.random.default_rng(5)
    logits = make(6, G, N, V, "f32") * 200 + 5000
    z = ou.as_float64(logits)
    scores = rng.normal(-3000, 20, G * N).astype(np.float32)
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    got = smcsd.beam_select(logits, G, N, V, M, scores=dev(scores), ws=ws)
    tokens, anc, score, _, gap = ou.beam_select(z, G, N, V, M, scores=scores)
    assert gap > 1e-8 and smcsd.check_status(ws) == 0
    assert np.array_equal(host(got["tokens"]).reshape(G, M), tokens) and np.array_equal(host(got["ancestors"]).reshape(G, M), anc)
    assert np.allclose(host(got["scores"]).reshape(G, M), score, rtol=2.0 ** -24, atol=2e-6)


def test_a_call_repeats_its_bits_and_runs_captured(smcsd):
    G, N, V, M = 4, 16, 32000, 16
    logits, scores = make(1, G, N, V, "bf16"), torch.linspace(-4, 0, G * N, device="cuda")
    want = smcsd.beam_select(logits, G, N, V, M, scores=scores)
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    out = {k: torch.empty_like(v) for k, v in want.items()}

    def call():
        smcsd.beam_select(logits, G, N, V, M, scores=scores, ws=ws, tokens=out["tokens"], ancestors=out["ancestors"], out_scores=out["scores"],
                          out_finished=out["finished"])
    for _ in range(20):
        call()
        assert all(torch.equal(out[k], want[k]) for k in want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    logits.copy_(make(2, G, N, V, "bf16"))
    want = smcsd.beam_select(logits, G, N, V, M, scores=scores)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want) and smcsd.check_status(ws) == 0


def test_draft_trees_children(smcsd):
    # a node's children and a tree's best nodes: one row's best, then the best of all the frontier's continuations
    V, W = 5000, 6
    first = make(1, 1, 1, V, "bf16")
    a = smcsd.beam_select(first, 1, 1, V, W)
    logits = make(2, 1, W, V, "bf16")
    b = smcsd.beam_select(logits, 1, W, V, W, scores=a["scores"])
    z0, z1 = torch.log_softmax(first.double(), 1), torch.log_softmax(logits.double(), 1)
    total = z0[0, a["tokens"].long()][:, None] + z1
    want = total.flatten().topk(W)
    assert torch.equal(b["ancestors"].long() * V + b["tokens"].long(), want.indices)
    assert (b["scores"].double() - want.values).abs().max() < 1e-5


def test_a_group_of_the_largest_size(smcsd):
    # 64 rows of 1.2 million logits: 37 500 chunks, whose scores fill the shared memory
    N, V, M = 64, 1_200_000, 48
    logits, scores = make(3, 1, N, V, "bf16"), torch.linspace(-2, 0, N, device="cuda")
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, N, 0, V)
    got = smcsd.beam_select(logits, 1, N, V, M, scores=scores, ws=ws)
    assert smcsd.check_status(ws) == 0
    x = torch.stack([torch.log_softmax(logits[i].double(), 0) for i in range(N)]).add_(scores.double()[:, None]).flatten()
    value = x.topk(M).values
    assert bool((value[:-1] - value[1:] >= 0).all())
    at = got["ancestors"].long() * V + got["tokens"].long()
    assert torch.equal(x[at], value)  # the same candidates in the same order (equal ones are of one row)
    same = value[:-1] == value[1:]
    assert bool((at[:-1] < at[1:])[same].all())
    assert float((got["scores"].double() - value).abs().max()) <= 2e-6 + 2.0 ** -24 * float(value.abs().max())
    with pytest.raises(smcsd.SMCSDError):
        smcsd.beam_select(logits[:, :1].contiguous(), 1, 64, 1, 257)
