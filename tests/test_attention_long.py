"""Attention over contexts that give every block of the kernels runs of many key tiles: loops over the rings, maxima that
move in the middle of a run, streams and groups of warps side by side, shares weighted by rows. Against the definition in 64
bits (torch, on the GPU), within the bounds of serve_util.attention_bounds.

Keys. Along one direction u of the queries most keys have a score near 0; in every third tile one key stands 7 (tile 2 of 6)
or 14 (tile 4 of 6) above them, times a factor of the row's own: 1, 0.5, 0 or -0.7. So any six tiles in a row raise a row's
maximum at least once by more than 8 log 2, some rows by less. Values are positive, and those of the high keys as much
smaller as their weights are larger: what was added up before a maximum moves is most of the result."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, host

pytestmark = pytest.mark.gpu

TILE, PAGE = 128, 16
LEVELS = {2: 7.0, 4: 14.0}
FACTORS = (1.0, 0.5, 0.0, -0.7)


class Long:
    def __init__(self, seed, ctx, counts, T, Hq, Hkv, D, dtype, N=1, shared=0, tree=False, scale=None, moving=True):
        rng, gen = np.random.default_rng(seed), torch.Generator("cuda").manual_seed(seed)
        S, R = len(ctx), int(sum(counts))
        P = max(1, max((c + n + PAGE - 1) // PAGE for c, n in zip(ctx, counts)))
        table = rng.permutation(S * P).astype(np.int32).reshape(S, P)
        for s in range(S):
            table[s, :shared // PAGE] = table[s // N * N, :shared // PAGE]
        self.scale = D ** -0.5 if scale is None else scale
        a = 16.0
        randn = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
        k, v = randn(S * P, Hkv, PAGE, D), 1 + 0.3 * randn(S * P, Hkv, PAGE, D)
        k[..., 0] = 0.0
        for s in range(S) if moving else ():
            for t in range(ctx[s] // TILE):
                level = LEVELS.get(t % 6)
                if level is None:
                    continue
                pos = t * TILE + int(rng.integers(TILE))
                page = int(table[s, pos // PAGE])
                k[page, :, pos % PAGE, 0] = level / (a * D ** -0.5)
                v[page, :, pos % PAGE] *= float(np.exp(-level))
        q = 0.3 * randn(R, Hq, D)
        q[..., 0] = a * torch.tensor(FACTORS, device="cuda")[torch.arange(R, device="cuda")[:, None].add(torch.arange(Hq, device="cuda")) % 4]
        if self.scale < 0:
            q = -q
        self.q, self.k, self.v = q.to(dtype), k.to(dtype), v.to(dtype)
        self.table, self.ctx, self.counts, self.T, self.N = table, list(ctx), list(counts), T, N
        self.S, self.R, self.Hq, self.Hkv, self.D, self.dtype = S, R, Hq, Hkv, D, dtype
        parents = su.random_parents(counts, rng) if tree else None
        self.lists = su.seen_lists(counts, parents)
        self.mask = dev(su.mask_words(counts, T, self.lists).view(np.int32)) if tree else None
        self.offsets = dev(su.offsets_of(counts)) if len(set(counts)) > 1 or counts[0] != T else None
        self.ws = None

    def run(self, smcsd):
        if self.ws is None:
            self.ws = smcsd.TreeAttentionWorkspace(self.S, self.N, self.T, self.Hq, self.Hkv, self.D)
        out, lse = torch.full_like(self.q, 7.0), torch.full((self.R, self.Hq), 7.0, device="cuda")
        smcsd.tree_attention(self.q, self.k, self.v, dev(self.table), dev(np.array(self.ctx, np.int32)), self.S, self.T, self.scale,
                             N=self.N, node_offsets=self.offsets, mask=self.mask, ws=self.ws, out=out, lse=lse)
        assert smcsd.check_status(self.ws) == 0
        return out, lse

    def exact(self):
        """out, lse, sum p |v|, largest sum |q k| |scale|, one sequence after the other."""
        parts, r = [], 0
        table = dev(self.table).long()
        for s, (c, n) in enumerate(zip(self.ctx, self.counts)):
            if n == 0:
                continue
            pos = torch.arange(c + n, device="cuda")
            pages = table[s, pos // PAGE]
            k, v = (x[pages, :, pos % PAGE].double() for x in (self.k, self.v))  # [keys, Hkv, D]
            q = self.q[r:r + n].double().unflatten(1, (self.Hkv, self.Hq // self.Hkv))
            seen = torch.zeros(n, c + n, dtype=torch.bool, device="cuda")
            seen[:, :c] = True
            for t in range(n):
                seen[t, c + torch.tensor(self.lists[r + t], device="cuda")] = True
            none, zero = torch.tensor([float("-inf"), 0.0], dtype=torch.float64, device="cuda")
            z = torch.where(seen[:, None, None], torch.einsum("nhgd,xhd->nhgx", q, k) * self.scale, none)
            reach = torch.where(seen[:, None, None], torch.einsum("nhgd,xhd->nhgx", q.abs(), k.abs()) * abs(self.scale), zero).amax(-1)
            m = z.amax(-1, keepdim=True)
            e = torch.exp(z - m)
            l = e.sum(-1, keepdim=True)
            p = e / l
            parts.append((torch.einsum("nhgx,xhd->nhgd", p, v).flatten(1, 2), (m + torch.log(l))[..., 0].flatten(1),
                          torch.einsum("nhgx,xhd->nhgd", p, v.abs()).flatten(1, 2), reach.flatten(1)))
            r += n
        return [host(torch.cat(x)) for x in zip(*parts)]

    def check(self, out, lse):
        want, wlse, spread, reach = self.exact()
        keys = max(c + n for c, n in zip(self.ctx, self.counts))
        bound, rel = su.attention_bounds(spread, reach, want, self.D, keys, self.dtype == torch.bfloat16)
        got, glse = host(out.double()), host(lse).astype(np.float64)
        off = np.abs(got - want)
        assert (off <= bound).all(), (float((off / bound).max()), np.argwhere(~(off <= bound))[:4])
        assert (np.abs(glse - wlse) <= rel + 2.0 ** -22 * (1 + np.abs(wlse) + reach)).all()

    def tiles(self, keys_per_tile, rows_per_block):
        """Key tiles of all units without groups."""
        g = self.Hq // self.Hkv
        return sum(self.Hkv * -(-n * g // rows_per_block) * -(-(c + n) // keys_per_tile) for c, n in zip(self.ctx, self.counts))


def run_and_check(smcsd, *a, **k):
    c = Long(*a, **k)
    out, lse = c.run(smcsd)
    c.check(out, lse)
    again, lse2 = c.run(smcsd)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    return c


BF16, F32 = torch.bfloat16, torch.float32
# rows of a unit: (T, query heads for each key head, D). Without groups the narrow kernel takes up to 96 rows (D = 128) or 64
ROWS = [(2, 4, 128), (8, 4, 128), (10, 4, 128), (16, 4, 128), (45, 2, 128), (24, 4, 128),  # narrow: 8, 32, 40, 64, 90, 96
        (50, 2, 128), (32, 4, 128), (25, 8, 128), (64, 4, 128), (75, 4, 128),              # wide: 100, 128, 200, 256, 300
        (3, 4, 64), (13, 3, 64), (16, 4, 64), (33, 2, 64), (43, 3, 64), (90, 3, 64)]       # 12, 39, 64 | 66, 129, 270


@pytest.mark.parametrize("T,g,D", ROWS)
@pytest.mark.parametrize("tree", [False, True])
def test_runs_of_many_tiles(smcsd, T, g, D, tree):
    counts = [T, T - T // 3]
    c = run_and_check(smcsd, T + D, [14801, 14500], counts, T, 4 * g, 4, D, BF16, tree=tree)
    assert c.tiles(TILE, 256) >= 6 * 152


@pytest.mark.parametrize("T,g,D", [(1, 4, 128), (10, 4, 64), (20, 2, 128)])
@pytest.mark.parametrize("tree", [False, True])
def test_runs_of_many_tiles_float32(smcsd, T, g, D, tree):
    c = run_and_check(smcsd, T, [14801, 15500], [T, T], T, 4 * g, 4, D, F32, tree=tree)
    assert c.tiles(64, 16) >= 6 * 2 * 152


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,g,D", [(2, 4, 128), (45, 2, 128), (50, 2, 128), (25, 8, 128), (3, 4, 64), (33, 2, 64)])
@pytest.mark.parametrize("scale", [-1.0, 0.0])
def test_negative_and_zero_scales(smcsd, dtype, T, g, D, scale):
    run_and_check(smcsd, 3 * T + D, [9000, 2100], [T, T], T, 4 * g, 4, D, dtype, scale=scale * D ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,g,D,N", [(5, 4, 128, 4), (8, 4, 128, 3), (12, 4, 128, 4), (4, 4, 64, 8), (9, 4, 64, 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_groups_over_long_shared_contexts(smcsd, dtype, T, g, D, N, tree):
    # shared units of many tiles, heavy and light ones on one line, and own units of a few to many tiles
    counts = [T - (s % 3 == 2) for s in range(2 * N)]
    ctx = [12000 + 700] * N + [9000 + 90] * N
    run_and_check(smcsd, T + N, ctx, counts, T, 4 * g, 4, D, dtype, N=N, shared=8960, tree=tree)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,T,g", [(64, 2, 2), (128, 60, 2)])
def test_more_sequences_than_a_warp_plans(smcsd, dtype, D, T, g):
    # the planning kernel without groups
    rng = np.random.default_rng(D)
    S = 1027
    counts = [int(x) for x in rng.integers(0, T + 1, S)]
    ctx = [int(x) for x in rng.integers(0, 300, S)]
    ctx[5], counts[5], ctx[1000], counts[1000] = 9000, T, 4000, T  # units that are cut
    run_and_check(smcsd, D, ctx, counts, T, 2 * g, 2, D, dtype, moving=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,g,D", [(10, 4, 128), (50, 2, 128), (25, 8, 128), (7, 4, 64)])
def test_nan_in_a_late_node_of_a_long_run(smcsd, dtype, bad, T, g, D):
    c = Long(T, [14801], [T], T, 8 * g, 8, D, dtype, tree=True)
    good, glse = c.run(smcsd)
    at = T // 2
    sees = torch.tensor([at in seen for seen in c.lists], device="cuda")
    pos = c.ctx[0] + at
    page = int(c.table[0, pos // PAGE])
    heads = slice(3 * g, 4 * g)
    other = torch.ones(c.Hq, dtype=torch.bool, device="cuda")
    other[heads] = False
    for cache in (c.v, c.k):
        kept = cache[page, 3, pos % PAGE, 2].clone()
        cache[page, 3, pos % PAGE, 2] = bad
        out, lse = c.run(smcsd)
        assert torch.equal(out[~sees], good[~sees]) and torch.equal(lse[~sees], glse[~sees])
        assert torch.equal(out[:, other], good[:, other]) and torch.equal(lse[:, other], glse[:, other])
        if cache is c.v:
            hit = out[sees][:, heads].float()
            assert bool((torch.isnan(hit[..., 2]) if bad != bad else hit[..., 2] == bad).all())
            rest = torch.arange(D, device="cuda") != 2
            assert torch.equal(hit[..., rest], good[sees][:, heads].float()[..., rest])
        cache[page, 3, pos % PAGE, 2] = kept
    out, lse = c.run(smcsd)
    assert torch.equal(out, good) and torch.equal(lse, glse)
