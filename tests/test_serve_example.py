"""The example's whole steps: what the cache, the tables and the counts hold after a few of them."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from gpu_util import host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "serve_step.py")
    spec = importlib.util.spec_from_file_location("serve_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("G,N,K,page,dtype", [
    (4, 8, 4, 16, torch.bfloat16), (3, 1, 2, 8, torch.bfloat16), (2, 16, 7, 32, torch.bfloat16), (2, 4, 3, 16, torch.float32)])
def test_steps(smcsd, example, G, N, K, page, dtype):
    session = example.Session(G=G, N=N, K=K, page=page, pages_per_seq=256 // page, dtype=dtype, seed=G + N)
    start = host(session.ctx).copy()
    for step in range(6):
        before = host(session.tokens)
        got = session.step()
        session.check()
        parent = np.arange(G * N) // N * N + host(got["ancestors"])
        ctx, tokens, table, ref = host(session.ctx), host(session.tokens), host(session.table), host(session.refcount)
        assert np.array_equal(ctx, start + (step + 1) * (K + 1))
        # a particle goes on from its parent's tokens, with K + 1 more
        for s in range(G * N):
            old = ctx[s] - K
            assert np.array_equal(tokens[s, :old], before[parent[s], :old])
            assert (tokens[s, :ctx[s] + 1] >= 0).all() and (tokens[s, ctx[s] + 1:] == -1).all()
        # the counts are those of the tables
        assert np.array_equal(ref, np.bincount(table[table >= 0].ravel(), minlength=ref.size))
        # every particle's pages hold the keys and values of its own tokens
        kv = session.qkv[torch.from_numpy(tokens).clamp(min=0).long().cuda()][:, :, session.Hq * session.D:]
        kv = kv.unflatten(2, (2, session.Hkv, session.D))
        for s in range(G * N):
            pages = session.table[s, :(ctx[s] + page - 1) // page].long()
            for i, cache in enumerate((session.k_cache, session.v_cache)):
                held = cache[pages].permute(0, 2, 1, 3).flatten(0, 1)[:ctx[s]]
                assert torch.equal(held, kv[s, :ctx[s], i]), (step, s, i)


def test_attention_of_a_step_is_that_of_the_particles_own_tokens(smcsd, example):
    # the table that a step leaves, read with and without groups, against the tokens' keys and values themselves
    session = example.Session(G=2, N=8, K=4, page=16, dtype=torch.float32, seed=3)
    for _ in range(4):
        session.step()
    S, D, Hq, Hkv = session.S, session.D, session.Hq, session.Hkv
    n = int(session.ctx[0])
    ctx = session.ctx - 1  # the last cached token as the only node
    q = session.qkv[session.tokens.gather(1, ctx[:, None].long())[:, 0].long()][:, :Hq * D].unflatten(1, (Hq, D)).contiguous()
    outs = [smcsd.tree_attention(q, session.k_cache, session.v_cache, session.table, ctx, S, 1, D ** -0.5, N=N)[0] for N in (1, 8)]
    for s in range(S):
        m = int(session.ctx[s])
        kv = session.qkv[session.tokens[s, :m].long()][:, Hq * D:].unflatten(1, (2, Hkv, D)).double()
        k, v = (kv[:, i].repeat_interleave(Hq // Hkv, 1) for i in range(2))
        z = torch.einsum("hd,xhd->hx", q[s].double(), k) * D ** -0.5
        want = torch.einsum("hx,xhd->hd", z.softmax(1), v)
        # float32: scores of 64 products and sums of up to m weights, each off by a few units of 2^-24 of what is added up
        reach = torch.einsum("hd,xhd->hx", q[s].double().abs(), k.abs()).amax() * D ** -0.5
        bound = (2 * (D + 8) * float(reach) + m + 16) * 2.0 ** -24 * float(v.abs().amax())
        for out in outs:
            assert float((out[s].double() - want).abs().amax()) <= bound
    assert n > 1
