"""Forks, freeing, compaction and copies of cache pages, and states by ancestors, against their rules one entry at a time."""
import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


def random_table(rng, S, P, num, fill=0.6):
    """Tables with shared pages, and counts with other holders."""
    have = rng.integers(0, P + 1, S)
    table = np.full((S, P), -1, np.int32)
    pool = rng.permutation(num)[:max(1, int(num * fill))]
    for s in range(S):
        table[s, :have[s]] = rng.choice(pool, have[s])
    ref = np.bincount(table[table >= 0].ravel(), minlength=num).astype(np.int32)
    ref[rng.random(num) < 0.1] += 1
    return table, ref


@pytest.mark.parametrize("S,P,num,page", [(1, 1, 1, 8), (4, 3, 7, 8), (16, 130, 3000, 16), (33, 17, 200, 32), (300, 64, 90_000, 16), (1024, 700, 50_000, 64)])
def test_fork_and_free(smcsd, S, P, num, page):
    rng = np.random.default_rng(S + P)
    table, ref = random_table(rng, S, P, num)
    parents = rng.integers(-1, S, S).astype(np.int32)
    stay = rng.random(S) < 0.4
    parents[stay] = np.arange(S)[stay]
    lengths = rng.integers(0, P * page + 2 * page, S).astype(np.int32)
    lengths[rng.random(S) < 0.2] = np.iinfo(np.int32).max
    lengths[:1] = 0
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    for par, length in ((parents, lengths), (parents, None), (np.arange(S, dtype=np.int32), lengths), (np.full(S, -1, np.int32), None)):
        want = ou.fork(table, ref, par, None if length is None else np.minimum(length, P * page), page)
        got = smcsd.kv_fork(dev(table), dev(ref), dev(par), page, lengths=None if length is None else dev(length), ws=ws)
        assert smcsd.check_status(ws) == 0
        assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    want = ou.fork(table, ref, None, np.minimum(lengths, P * page), page)
    got = smcsd.kv_free(dev(table), dev(ref), dev(lengths), page, ws=ws)
    assert smcsd.check_status(ws) == 0
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])


@pytest.mark.parametrize("S,P", [(3, 30_001), (70, 1027), (70, 1028), (33, 2052), (20, 4096), (300, 300), (20_000, 4), (20_000, 5)])
@pytest.mark.parametrize("shift", [0, 1])
def test_large_tables_of_every_row_and_address(smcsd, S, P, shift):
    rng = np.random.default_rng(S + P)
    num, page = 70_001, 16
    table, ref = random_table(rng, S, P, num)
    parents = np.where(rng.random(S) < 0.4, np.arange(S), rng.integers(-1, S, S)).astype(np.int32)
    lengths = rng.integers(0, P * page + 1, S).astype(np.int32)
    flat = dev(np.concatenate([np.zeros(shift, np.int32), table.ravel()]))[shift:].view(S, P)  # off the vectors' addresses
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    want = ou.fork(table, ref, parents, lengths, page)
    got = smcsd.kv_fork(flat, dev(ref), dev(parents), page, lengths=dev(lengths), ws=ws)
    assert smcsd.check_status(ws) == 0
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])


@pytest.mark.parametrize("G,N,P,num", [(1, 1, 1, 1), (1, 4, 33, 200), (3, 5, 100, 1500), (4, 8, 128, 4096), (8, 8, 128, 8192), (8, 8, 129, 8192), (2, 4, 10, 9000)])
def test_pagetable_remap_of_every_size(smcsd, G, N, P, num):
    rng = np.random.default_rng(G + P)
    table = rng.integers(-1, num, (G * N, P)).astype(np.int32)
    anc = rng.integers(0, N, G * N).astype(np.int32)
    resampled = rng.integers(0, 2, G).astype(np.int32)
    ws = smcsd.Workspace(smcsd.OP_PAGETABLE_REMAP, G)
    for res in (None, resampled):
        group = np.arange(G * N) // N
        row = group * N + (anc if res is None else np.where(res[group] != 0, anc, np.arange(G * N) % N))
        want = table[row]
        got, count = smcsd.kv_pagetable_remap(dev(anc), None if res is None else dev(res), G, N, dev(table), P, num, ws=ws)
        assert smcsd.check_status(ws) == 0
        assert np.array_equal(host(got), want) and np.array_equal(host(count), np.bincount(want[want >= 0].ravel(), minlength=num))
    table[0, 0] = num
    anc[-1] = N
    smcsd.kv_pagetable_remap(dev(anc), None, G, N, dev(table), P, num, ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_RANGE


def test_fork_reads_the_old_table(smcsd):
    # two sequences change places, a third follows one of them
    table = np.array([[0, 1, -1], [2, -1, -1], [3, 4, 5]], np.int32)
    ref = np.ones(8, np.int32)
    ref[6:] = 0
    got, count = smcsd.kv_fork(dev(table), dev(ref), dev(np.array([1, 0, 0], np.int32)), 16)
    assert host(got).tolist() == [[2, -1, -1], [0, 1, -1], [0, 1, -1]]
    assert host(count).tolist() == [2, 2, 1, 0, 0, 0, 0, 0]


def test_one_prompt_forked_into_many_and_freed_again(smcsd):
    S, P, page = 64, 256, 16
    table = np.full((S, P), -1, np.int32)
    table[5, :200] = np.random.default_rng(0).permutation(1000)[:200]
    ref = np.bincount(table[5, :200], minlength=1000).astype(np.int32)
    a, count = smcsd.kv_fork(dev(table), dev(ref), dev(np.full(S, 5, np.int32)), page, lengths=dev(np.full(S, 100 * page - 3, np.int32)))
    want = ou.fork(table, ref, np.full(S, 5), np.full(S, 100 * page - 3), page)
    assert np.array_equal(host(a), want[0]) and np.array_equal(host(count), want[1]) and host(count).max() == S
    b, count = smcsd.kv_free(a, count, dev(np.zeros(S, np.int32)), page)
    assert (host(b) == -1).all() and (host(count) == 0).all()


def test_bad_parents_lengths_and_pages(smcsd):
    table = np.array([[0, 1], [2, -1], [3, 9]], np.int32)
    ref = np.array([1, 1, 1, 1, 0, 0], np.int32)
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    bad = smcsd.ERR_RANGE
    for parents, lengths in (([3, 1, 2], None), ([-2, 1, 2], None), ([0, 1, 2], [-1, 32, 32])):
        t = table.copy()
        t[2, 1] = -1
        got, count = smcsd.kv_fork(dev(t), dev(ref), dev(np.array(parents, np.int32)), 16, ws=ws,
                                   lengths=None if lengths is None else dev(np.array(lengths, np.int32)))
        assert smcsd.check_status(ws) == bad
        assert np.array_equal(host(got), t) and np.array_equal(host(count), ref)  # kept as they are
    got, count = smcsd.kv_fork(dev(table), dev(ref), dev(np.arange(3, dtype=np.int32)), 16, ws=ws)  # a page that the cache does not have
    assert smcsd.check_status(ws) == bad and np.array_equal(host(got), table) and np.array_equal(host(count), ref)
    table[2, 1] = 4  # held, but counted by nobody
    smcsd.kv_free(dev(table), dev(ref), dev(np.zeros(3, np.int32)), 16, ws=ws)
    assert smcsd.check_status(ws) == bad


SIZES = [1, 2, 3, 31, 32, 33, 64, 1000, 4096, 4097, 33_000, 100_000, 300_001]


@pytest.mark.parametrize("num", SIZES)
@pytest.mark.parametrize("kind", ["mixed", "full", "none", "front", "back", "half"])
def test_compact(smcsd, num, kind):
    rng = np.random.default_rng(num)
    ref = dict(mixed=rng.integers(0, 3, num), full=np.ones(num), none=np.zeros(num), front=np.arange(num) < num // 3,
               back=np.arange(num) >= num - num // 3, half=np.arange(num) % 2)[kind].astype(np.int32)
    S, P = 7, 50
    held = np.nonzero(ref)[0]
    table = np.full((S, P), -1, np.int32)
    if held.size:
        table = np.where(rng.random((S, P)) < 0.8, rng.choice(held, (S, P)), -1).astype(np.int32)
    want = ou.compact(table, ref)
    ws = smcsd.Workspace(smcsd.OP_KV_COMPACT, 1, 0, num)
    got = smcsd.kv_compact(dev(table), dev(ref), ws=ws)
    assert smcsd.check_status(ws) == 0
    n = want[2].size
    assert host(got["counts"]).tolist() == [n, want[4]]
    assert np.array_equal(host(got["table_out"]), want[0]) and np.array_equal(host(got["refcount_out"]), want[1])
    src, dst = host(got["src"]), host(got["dst"])
    assert src.size == dst.size == num // 2
    assert np.array_equal(src[:n], want[2]) and np.array_equal(dst[:n], want[3]) and (src[n:] == -1).all() and (dst[n:] == -1).all()
    # what is compact stays
    again = smcsd.kv_compact(got["table_out"], got["refcount_out"], ws=ws)
    assert host(again["counts"]).tolist() == [0, want[4]] and torch.equal(again["table_out"], got["table_out"])


def test_compact_reports_tables_and_counts_that_do_not_fit(smcsd):
    ws = smcsd.Workspace(smcsd.OP_KV_COMPACT, 1, 0, 6)
    ref = np.array([0, 1, 0, 0, 1, 0], np.int32)
    for entry in (6, -2, 0):  # outside, and a free page
        table = np.array([[1, 4, entry]], np.int32)
        got = smcsd.kv_compact(dev(table), dev(ref), ws=ws)
        assert smcsd.check_status(ws) == smcsd.ERR_RANGE
        assert host(got["table_out"]).tolist() == [[1, 0, entry]]
    ref[3] = -1
    got = smcsd.kv_compact(dev(np.array([[1, 4]], np.int32)), dev(ref), ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_RANGE
    assert host(got["refcount_out"]).tolist() == [1, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("shape,dtype,layers", [((9, 1, 8, 1), torch.float16, 1), ((40, 2, 16, 64), torch.bfloat16, 2), ((33, 3, 8, 100), torch.float32, 3),
                                                ((700, 8, 16, 128), torch.bfloat16, 4), ((12, 8, 256, 128), torch.float32, 1)])
def test_copy_pages(smcsd, shape, dtype, layers):
    rng = np.random.default_rng(shape[0])
    num = shape[0]
    caches = [torch.randn(shape, device="cuda").to(dtype) for _ in range(2 * layers)]
    order = rng.permutation(num)
    n = num // 2 - 1
    src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
    src[0] = dst[0] = -1
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    for count in (None, 0, 1, n // 2, n):
        want = [c.clone() for c in caches]
        upto = n if count is None else count
        for c in want:
            for a, b in zip(src[:upto], dst[:upto]):
                if a >= 0:
                    c[b] = c[a]
        got = smcsd.kv_copy_pages(caches, dev(src), dev(dst), count=None if count is None else dev(np.array([count, 5], np.int32)), ws=ws)
        assert smcsd.check_status(ws) == 0 and got is caches
        assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_copies_out_of_range_write_nothing(smcsd):
    cache = torch.randn(5, 1, 8, 64, device="cuda")
    want = cache.clone()
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    for src, dst, count in (([5], [0], None), ([0], [5], None), ([-1], [2], None), ([2], [-1], None), ([0, 1], [2, 3], 3), ([0], [2], -1)):
        smcsd.kv_copy_pages([cache], dev(np.array(src, np.int32)), dev(np.array(dst, np.int32)), ws=ws,
                            count=None if count is None else dev(np.array([count], np.int32)))
        assert smcsd.check_status(ws) == smcsd.ERR_RANGE
        assert torch.equal(cache, want)


def test_copies_past_four_gigabytes(smcsd):
    cache = torch.zeros(1100, 8, 256, 1024, device="cuda", dtype=torch.bfloat16)  # 4.6 GB, pages of 4 MB
    page = torch.randn(cache.shape[1:], device="cuda").bfloat16()
    cache[1] = page
    smcsd.kv_copy_pages([cache], dev(np.array([1], np.int32)), dev(np.array([1099], np.int32)))
    smcsd.kv_copy_pages([cache], dev(np.array([1099], np.int32)), dev(np.array([1040], np.int32)))
    assert torch.equal(cache[1099], page) and torch.equal(cache[1040], page) and int(cache[1098].count_nonzero()) == 0


@pytest.mark.parametrize("G,N,M", [(1, 1, 1), (3, 4, 4), (2, 16, 16), (5, 1, 7), (2, 8, 3), (1, 300, 300)])
def test_state_reorder(smcsd, G, N, M):
    rng = np.random.default_rng(G + N + M)
    S = G * N
    anc = rng.integers(0, N, G * M).astype(np.int32)
    states = [torch.randn(S, 33, device="cuda"), torch.randn(S, 2048, device="cuda").bfloat16(), torch.rand(S, device="cuda"),
              torch.randint(0, 100, (S, 5, 3), device="cuda", dtype=torch.uint8), torch.randint(0, 9, (S, 4), device="cuda"),
              torch.rand(S, 7, device="cuda") < 0.5, torch.randn(S, 3, device="cuda").half(), torch.randn(S, 100_000, device="cuda")]
    parent = torch.from_numpy(np.repeat(np.arange(G), M) * N + anc).cuda()
    ws = smcsd.Workspace(smcsd.OP_STATE_REORDER, 1)
    got = smcsd.state_reorder(states, dev(anc), G, N, M, ws=ws)
    assert smcsd.check_status(ws) == 0 and len(got) == len(states)
    for a, s in zip(got, states):
        assert a.dtype == s.dtype and torch.equal(a, s[parent])
    out = [torch.zeros_like(a) for a in got]
    back = smcsd.state_reorder(tuple(states), dev(anc), G, N, M, out=out, ws=ws)
    for a, b, c in zip(back, out, got):
        assert a.data_ptr() == b.data_ptr() and torch.equal(a, c)


def test_ancestors_out_of_range_leave_their_rows(smcsd):
    state = torch.arange(12, device="cuda", dtype=torch.float32).view(6, 2)
    ws = smcsd.Workspace(smcsd.OP_STATE_REORDER, 1)
    for bad in (3, -1, 2 ** 31 - 1, -2 ** 31):
        out = torch.full((6, 2), -5.0, device="cuda")
        smcsd.state_reorder([state], dev(np.array([0, bad, 2, 1, 1, 0], np.int32)), 2, 3, out=[out], ws=ws)
        assert smcsd.check_status(ws) == smcsd.ERR_RANGE
        want = state[torch.tensor([0, 0, 2, 4, 4, 3])]
        want[1] = -5.0
        assert torch.equal(out, want)


def test_captured_together(smcsd):
    rng = np.random.default_rng(3)
    S, P, num, page = 16, 20, 500, 16
    table, ref = random_table(rng, S, P, num)
    cache = [torch.randn(num, 2, page, 64, device="cuda") for _ in range(2)]
    lengths, parents = rng.integers(0, P * page, S).astype(np.int32), rng.integers(-1, S, S).astype(np.int32)
    t, r, n, p = dev(table), dev(ref), dev(lengths), dev(parents)
    ws = smcsd.Workspace(smcsd.OP_KV_COMPACT, 1, 0, num)

    def step():
        a = smcsd.kv_free(t, r, n, page, ws=ws)
        b = smcsd.kv_fork(*a, p, page, ws=ws)
        c = smcsd.kv_compact(*b, ws=ws)
        smcsd.kv_copy_pages(cache, c["src"], c["dst"], count=c["counts"], ws=ws)
        return c
    start = [c.clone() for c in cache]
    step()
    first = [c.clone() for c in cache]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c = step()
    for a, b in zip(cache, start):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    freed = ou.fork(table, ref, None, lengths, page)
    want = ou.compact(*ou.fork(*freed, parents, None, page))
    assert np.array_equal(host(c["table_out"]), want[0]) and np.array_equal(host(c["refcount_out"]), want[1])
    assert all(torch.equal(a, b) for a, b in zip(cache, first)) and smcsd.check_status(ws) == 0
