"""Attention of drafted tokens over a paged cache against a plain float64 form, within bounds that
follow from the arithmetic (serve_util.attention_bounds)."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    """A cache with every position that no row sees set to NaN, and queries as slices of wider rows."""

    def __init__(self, seed, ctx, counts, T, Hq, Hkv, D, page, dtype, N=1, shared=0, parents=None, std=2.0, pool=0):
        rng = np.random.default_rng(seed)
        torch.manual_seed(seed)
        S, R = len(ctx), int(sum(counts))
        P = max(1, max((c + n + page - 1) // page for c, n in zip(ctx, counts))) + 1
        num = S * P + pool
        table = rng.permutation(num)[: S * P].astype(np.int32).reshape(S, P)
        for s in range(S):  # the first `shared` tokens' full pages are those of the group's first sequence
            k = min(shared, ctx[s]) // page
            table[s, :k] = table[s // N * N, :k]
        live = np.zeros((num, page), bool)
        for s in range(S):
            pos = np.arange(ctx[s] + counts[s])
            live[table[s, pos // page], pos % page] = True
            table[s, (ctx[s] + counts[s] + page - 1) // page:] = -1
        live = torch.from_numpy(live).cuda()[:, None, :, None]
        nan = torch.full((), float("nan"), device="cuda")
        self.k, self.v = (torch.where(live, torch.randn(num, Hkv, page, D, device="cuda"), nan).to(DT[dtype])
                          for _ in range(2))
        self.wide = torch.randn(R, Hq + 3, D, device="cuda").mul(std).to(DT[dtype])
        self.q = self.wide[:, 2: 2 + Hq]
        self.table, self.ctx, self.counts, self.T, self.N, self.D = table, list(ctx), list(counts), T, N, D
        self.Hq, self.Hkv, self.dtype, self.scale = Hq, Hkv, dtype, 1.0 / np.sqrt(D)
        self.parents = parents
        self.lists = su.seen_lists(counts, parents)
        self.words = None if parents is None else su.mask_words(counts, T, self.lists)

    def run(self, smcsd, ragged=None, stream=None):
        S = len(self.ctx)
        ragged = len(set(self.counts)) > 1 or self.counts[0] != self.T if ragged is None else ragged
        ws = smcsd.TreeAttentionWorkspace(S, self.N, self.T, self.Hq, self.Hkv, self.D)
        mask = None if self.words is None else dev(self.words.view(np.int32))
        off = dev(su.offsets_of(self.counts)) if ragged else None
        args = (self.q, self.k, self.v, dev(self.table), dev(np.array(self.ctx, np.int32)), S, self.T, self.scale)
        for _ in range(2):  # the workspace serves call after call
            out, lse = smcsd.tree_attention(*args, N=self.N, node_offsets=off, mask=mask, ws=ws, stream=stream)
        assert smcsd.check_status(ws, stream) == 0
        return out, lse

    def check(self, out, lse):
        f = lambda t: host(t.float()).astype(np.float64)  # noqa: E731
        want, wlse, spread, reach = su.attention(f(self.q), f(self.k), f(self.v), self.table, self.ctx, self.counts,
                                                 self.lists, self.scale)
        keys = max(c + n for c, n in zip(self.ctx, self.counts))
        bound, rel = su.attention_bounds(spread, reach, want, self.D, keys, self.dtype == "bf16")
        got, glse = f(out), host(lse).astype(np.float64)
        assert np.isfinite(got).all()
        off = np.abs(got - want)
        assert (off <= bound).all(), (float((off / bound).max()), np.argwhere(off > bound)[:4])
        none = np.isneginf(wlse)
        assert np.array_equal(none, np.isneginf(glse))
        # log of a sum that is off by rel, of a float32 sum of two terms
        lim = rel + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, wlse)) + reach)
        assert (np.abs(np.where(none, 0, glse) - np.where(none, 0, wlse)) <= lim).all()


def check(smcsd, *a, **k):
    c = Case(*a, **k)
    c.check(*c.run(smcsd))
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,T,Hq,Hkv,page", [
    ([0], 1, 1, 1, 8), ([1], 1, 4, 1, 16), ([0, 5], 3, 2, 2, 16), ([127, 128, 129], 1, 8, 2, 16), ([63, 64, 65], 2, 8, 8, 32),
    ([300, 1, 0, 517], 5, 8, 2, 8), ([255, 256], 4, 5, 5, 64), ([1000], 9, 16, 2, 256), ([40], 33, 16, 2, 16)])
def test_chains(smcsd, dtype, D, ctx, T, Hq, Hkv, page):
    check(smcsd, 7 * T + D, ctx, [T] * len(ctx), T, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hkv,page", [(2, 4, 2, 16), (31, 4, 4, 16), (64, 8, 1, 16), (65, 10, 2, 8), (130, 4, 2, 32)])
def test_ragged_trees(smcsd, dtype, T, Hq, Hkv, page):
    rng = np.random.default_rng(T)
    counts = [T, int(rng.integers(1, T + 1)), 1, int(rng.integers(1, T + 1))]
    ctx = [int(x) for x in rng.integers(0, 400, 4)]
    check(smcsd, T, ctx, counts, T, Hq, Hkv, 64, page, dtype, parents=su.random_parents(counts, rng))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sequence_without_nodes(smcsd, dtype):
    check(smcsd, 3, [50, 60, 70], [2, 0, 3], 3, 4, 2, 64, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,Hq,Hkv,shared,ctx", [
    (4, 1, 4, 2, 256, [300, 300, 520, 520]), (16, 5, 8, 2, 512, [700]), (3, 2, 5, 5, 1000, [128, 1001]), (8, 4, 32, 1, 384, [400]),
    (2, 1, 1, 1, 4, [9]), (64, 1, 8, 1, 640, [650])])
def test_groups_that_share_pages(smcsd, dtype, N, T, Hq, Hkv, shared, ctx):
    ctx = [c for c in ctx for _ in range(N)]
    c = check(smcsd, N + T, ctx, [T] * len(ctx), T, Hq, Hkv, 128, 16, dtype, N=N, shared=shared)
    c.N = 1  # and without the grouping
    c.check(*c.run(smcsd))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_of_ragged_trees(smcsd, dtype):
    rng = np.random.default_rng(8)
    counts = [int(x) for x in rng.integers(1, 12, 12)]
    check(smcsd, 8, [270] * 4 + [40] * 4 + [600] * 4, counts, 12, 6, 2, 64, 16, dtype, N=4, shared=260,
          parents=su.random_parents(counts, rng))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_that_leave_rows_empty(smcsd, dtype):
    c = Case(5, [0, 20, 0], [4, 4, 4], 4, 4, 2, 64, 16, dtype)
    c.words = np.array([[0], [1], [0], [15], [0], [0], [2], [0xFFFFFFFF], [8], [0], [0xFFFFFFF0], [4]], np.uint32)
    c.lists = su.seen_lists(c.counts, mask=c.words)
    out, lse = c.run(smcsd)
    c.check(out, lse)
    for r in (0, 2, 9, 10):  # no context and no node
        assert bool((out[r] == 0).all()) and bool(torch.isneginf(lse[r]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("T,ctx", [(6, 30), (40, 100), (140, 0)])
def test_nan_and_infinities_in_nodes_reach_their_own_rows_only(smcsd, dtype, bad, T, ctx):
    rng = np.random.default_rng(T)
    parents = su.random_parents([T], rng)
    c = Case(T, [ctx], [T], T, 8, 2, 64, 16, dtype, parents=parents)
    at = T // 2
    pos = ctx + at
    page = int(c.table[0, pos // 16])
    clean_k, clean_v = c.k.clone(), c.v.clone()
    sees = np.array([at in p for p in c.lists])
    for cache in ("v", "k"):
        c.k, c.v = clean_k.clone(), clean_v.clone()
        getattr(c, cache)[page, 1, pos % 16, 3] = float(bad)
        out, lse = c.run(smcsd)
        hit = torch.from_numpy(sees).cuda()
        c.k, c.v = clean_k, clean_v
        good, glse = c.run(smcsd)
        # other rows, and the other key head's: as if nothing had happened
        assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], glse[~hit])
        assert torch.equal(out[:, :4], good[:, :4])
        own = out[hit][:, 4:].float()
        if cache == "v":
            want = float(bad)
            col = own[..., 3]
            assert bool(torch.isnan(col).all()) if bad == "nan" else bool((col == want).all())
            assert bool(torch.isfinite(own[..., 4:]).all())


def test_infinite_keys_of_the_context(smcsd):
    # +inf or NaN scores make a row NaN, -inf scores are weights of zero: as the definition has it
    c = Case(9, [64], [2], 2, 2, 2, 64, 16, "bf16", std=1.0)
    c.k[int(c.table[0, 0]), :, 5] = float("inf")
    q = torch.zeros_like(c.wide)
    q[..., 0] = -1.0
    c.q = q[:, 2:4]
    c.k[int(c.table[0, 0]), :, 5, 1:] = 0.0
    out, lse = c.run(smcsd)  # the score of key 5 is -inf
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    c.q = -c.q
    out, lse = c.run(smcsd)
    assert bool(torch.isnan(out.float()).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(smcsd, dtype):
    check(smcsd, 4, [500, 200], [3, 3], 3, 4, 2, 64, 16, dtype, std=60.0)


def test_offsets_past_32_bits(smcsd):
    # pages whose elements lie past 2^31 and whose bytes lie past 2^32
    page, Hkv, D = 64, 4, 128
    num = (1 << 31) // (page * Hkv * D) + 64
    small = Case(2, [150], [3], 3, 8, Hkv, D, page, "bf16")
    big_k = torch.empty(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    big_v = torch.empty_like(big_k)
    ids = [num - 1 - 7 * j for j in range(3)]
    for j, i in enumerate(ids):
        big_k[i], big_v[i] = small.k[int(small.table[0, j])], small.v[int(small.table[0, j])]
    want, wlse = small.run(smcsd)
    table = small.table.copy()
    table[0, :3] = ids
    small.k, small.v, small.table = big_k, big_v, table
    out, lse = small.run(smcsd)
    assert torch.equal(out, want) and torch.equal(lse, wlse)


def test_another_stream_and_repeated_calls_agree(smcsd):
    c = Case(12, [333] * 8, [5] * 8, 5, 8, 2, 128, 16, "bf16", N=4, shared=320)
    a, la = c.run(smcsd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b, lb = c.run(smcsd, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_a_graph_replays_with_new_lengths(smcsd):
    c = Case(13, [700, 350], [4, 4], 4, 8, 2, 64, 16, "bf16")
    ws = smcsd.TreeAttentionWorkspace(2, 1, 4, 8, 2, 64)
    table, ctx = dev(c.table), dev(np.array([700, 350], np.int32))
    out, lse = torch.empty_like(c.q).contiguous(), torch.empty(8, 8, device="cuda")
    call = lambda: smcsd.tree_attention(c.q, c.k, c.v, table, ctx, 2, 4, c.scale, ws=ws, out=out, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([700, 350], [100, 350], [3, 0]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.ctx = lens
        c.check(out, lse)
    assert smcsd.check_status(ws) == 0


def test_errors_on_the_device(smcsd):
    c = Case(1, [40, 40], [2, 2], 2, 4, 2, 64, 16, "bf16")
    ws = smcsd.TreeAttentionWorkspace(2, 1, 2, 4, 2, 64)

    def status(table=c.table, ctx=(40, 40), off=None):
        smcsd.tree_attention(c.q, c.k, c.v, dev(table), dev(np.array(ctx, np.int32)), 2, 2, c.scale, ws=ws,
                             node_offsets=None if off is None else dev(np.array(off, np.int32)))
        return smcsd.check_status(ws)

    assert status() == 0
    assert status(ctx=(40, -1)) == smcsd.ERR_RANGE
    assert status(ctx=(40, 1000)) == smcsd.ERR_RANGE
    for bad in (-1, c.k.shape[0]):
        t = c.table.copy()
        t[1, 1] = bad
        assert status(table=t) == smcsd.ERR_RANGE
    for off in ([0, 3, 4], [0, -1, 4], [0, 2, 9], [0, 2, 1]):
        assert status(off=off) == smcsd.ERR_RANGE
    assert status() == 0
