"""beam_select where scores leave float32's range or cancel: tokens masked with the type's lowest value, scores above zero."""
import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


def best(z, G, N, M, T, scores, pad):
    """Tokens, ancestors, scores and flags by the definition. A candidate's score is kept as two float64, what is far below anything
    else and the rest, since one cannot hold both; a score that is minus infinity in float32 is no candidate's."""
    c = 1.0 / float(np.float32(T))
    top = z.max(1, keepdims=True)
    base = (0.0 if scores is None else scores.astype(np.float64)[:, None]) - np.log(np.exp((z - top) * c).sum(1, keepdims=True))
    far = z < -1e38
    high, low = np.where(far, z * c, 0.0), np.where(far, -top * c, (z - top) * c) + base
    with np.errstate(over="ignore"):
        there = ~np.isneginf((high + low).astype(np.float32))
    tokens, anc, out, over = np.full((G, M), pad), np.zeros((G, M), int), np.full((G, M), ou.NEG), np.ones((G, M), int)
    for g in range(G):
        beam, token = np.nonzero(there[g * N:(g + 1) * N])
        h, v = high[g * N + beam, token], low[g * N + beam, token]
        order = np.lexsort((token, beam, -v, -h))
        near = np.diff(v[order[:M + 1]])[(np.diff(beam[order[:M + 1]]) != 0) & (np.diff(h[order[:M + 1]]) == 0)]
        assert not ((np.abs(near) < 1e-8) & (near != 0)).any()  # the order is certain in float64
        order = order[:M]
        n = order.size
        tokens[g, :n], anc[g, :n], out[g, :n], over[g, :n] = token[order], beam[order], (h + v)[order], 0
    return tokens, anc, out, over


def check(smcsd, logits, G, N, V, M, T, scores=None, pad=7):
    """Against the definition. Scores within the error of one sum (1.9e-6) and half a step of float32."""
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    got = smcsd.beam_select(logits, G, N, V, M, temperature=T, scores=None if scores is None else dev(scores), pad_token=pad, ws=ws)
    assert smcsd.check_status(ws) == 0
    tokens, anc, want, over = best(ou.as_float64(logits), G, N, M, T, scores, pad)
    mine = host(got["scores"]).reshape(G, M).astype(np.float64)
    assert not np.isnan(mine).any()
    assert np.array_equal(host(got["tokens"]).reshape(G, M), tokens)
    assert np.array_equal(host(got["ancestors"]).reshape(G, M), anc)
    assert np.array_equal(host(got["finished"]).reshape(G, M), over)
    assert np.array_equal(np.isneginf(mine), np.isneginf(want))
    some = np.isfinite(want)
    assert (np.abs(mine[some] - want[some]) <= 2e-6 + 2.0 ** -24 * np.abs(want[some])).all()
    return mine


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [0.75, 0.25, 1.0, 2.0])
@pytest.mark.parametrize("G,N,V,M", [(5, 1, 1003, 20), (400, 1, 70, 12), (4, 3, 1003, 40), (310, 2, 70, 20), (1, 1, 40_000, 200), (1, 4, 9001, 200)])
def test_tokens_masked_with_the_lowest_value(smcsd, dtype, T, G, N, V, M):
    """Fewer tokens are left than are selected. With T below 1 a masked token's score lies below float32's range: it is none, whatever
    the number of beams."""
    t = ou.DTYPES[dtype]
    gen = torch.Generator("cuda").manual_seed(V + M)
    keep = 4
    logits = torch.full((G * N, V), torch.finfo(t).min, device="cuda", dtype=t)
    at = torch.rand(G * N, V, device="cuda", generator=gen).topk(keep, 1).indices
    logits.scatter_(1, at, (torch.randn(G * N, keep, device="cuda", generator=gen) * 3).to(t))
    scores = None if N == 1 else np.random.default_rng(M).normal(-5, 1, G * N).astype(np.float32)
    mine = check(smcsd, logits, G, N, V, M, T, scores)
    assert np.isfinite(mine).sum(1).max() == (min(M, N * keep) if T < 1 else min(M, N * V))


@pytest.mark.parametrize("N", [1, 3])
def test_scores_next_to_the_end_of_the_range(smcsd, N):
    """A beam whose own score is nearly as low as a float can be: its continuations fall out of the range one by one."""
    V, M = 500, 60 * N
    logits = torch.randn(N, V, device="cuda", generator=torch.Generator("cuda").manual_seed(N)) * 1e37
    scores = np.full(N, -3.3e38, np.float32)
    mine = check(smcsd, logits, 1, N, V, M, 1.0, scores)
    assert np.isneginf(mine).any() and np.isfinite(mine).any()


def beams_that_cancel(seed, N=64, each=16):
    """One group: beams with scores of 1e5, as bonuses make them, and a temperature that takes them back. But for one likely token a beam, all
    candidates' scores lie near zero, 1e-4 and more apart, though z less the row's maximum is rounded in steps of 7.6e-3 / c. One token
    in 64 is a candidate of any use, so that each stands in a range of its own."""
    f4 = np.float32
    rng = np.random.default_rng(seed)
    T = f4(0.001)
    c = 1.0 / float(T)
    step = 2.0 ** -17 * c  # of the scores of tokens next to one another
    z, scores = np.full((N, 64 * each), -130.0, f4), np.zeros(N, f4)
    for i in range(N):
        scores[i], top = f4(1e5 + rng.uniform(-300, 300)), f4(rng.uniform(0.2, 0.24))
        while abs((float(scores[i]) - c * float(top)) % step - (i + 0.5) * step / N) > 0.2 * step / N:
            top = np.nextafter(top, f4(4))
        k = np.floor((float(scores[i]) - c * float(top)) / step) + np.arange(each) - each // 2
        z[i, 17::64] = -(k * 2.0 ** -17)[rng.permutation(each)]
        z[i, 5] = top
    return z, scores, float(T)


@pytest.mark.parametrize("seed", [0, 14, 18])
def test_scores_that_cancel(smcsd, seed):
    z, scores, T = beams_that_cancel(seed)
    for M in range(66, 112):
        check(smcsd, torch.from_numpy(z).cuda(), 1, len(scores), z.shape[1], M, T, scores)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 700, 9001])
@pytest.mark.parametrize("G", [3, 310])
def test_sure_tokens_and_finished_beams_of_one_score(smcsd, dtype, V, G):
    """Beams with one token left, which has probability 1, keep their score, as finished beams do: equal scores go by the beam."""
    N, M = 6, 5
    rng = np.random.default_rng(V)
    z = np.full((G * N, V), ou.NEG)
    token = rng.integers(0, V, G * N)
    z[np.arange(G * N), token] = rng.normal(0, 3, G * N)
    if V > 2:  # far less likely ones in some rows: 2^-100 and below is nothing beside 1
        z[::4, :] = np.maximum(z[::4, :], -900.0)
    scores = np.repeat(rng.normal(-4, 1, G), N).astype(np.float32)
    finished = (rng.random(G * N) < 0.5).astype(np.int32)
    logits = torch.from_numpy(z).cuda().to(ou.DTYPES[dtype])
    ws = smcsd.Workspace(smcsd.OP_BEAM_SELECT, G * N, 0, V)
    got = smcsd.beam_select(logits, G, N, V, M, scores=dev(scores), finished=dev(finished), pad_token=V, ws=ws)
    assert smcsd.check_status(ws) == 0
    assert np.array_equal(host(got["ancestors"]).reshape(G, M), np.tile(np.arange(M), (G, 1)))
    assert np.array_equal(host(got["scores"]).reshape(G, M), scores.reshape(G, N)[:, :M])
    assert np.array_equal(host(got["tokens"]).reshape(G, M), np.where(finished, V, token).reshape(G, N)[:, :M])
    assert np.array_equal(host(got["finished"]).reshape(G, M), finished.reshape(G, N)[:, :M])
