"""Page tables, slots, cache writes and node masks against plain forms: whole numbers, equal."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


def shared_tables(rng, G, N, ctx, T, page, spare=0):
    """Tables of groups after a resampling: rows are copies of random ancestors' rows."""
    S = G * N
    P = (max(ctx) + T + page - 1) // page + 1
    num = S * P + spare
    own = rng.permutation(num)[: S * P].astype(np.int32).reshape(S, P)
    table = np.full((S, P), -1, np.int32)
    for s in range(S):
        a = s // N * N + int(rng.integers(N))
        have = (ctx[s] + page - 1) // page
        table[s, :have] = own[a, :have]
    ref = np.bincount(table[table >= 0].ravel(), minlength=num).astype(np.int32)
    return table, ref


def run_slots(smcsd, ctx, counts, T, table, ref, page, ragged, ws=None, stream=None):
    S = len(ctx)
    ws = ws or smcsd.Workspace(smcsd.OP_KV_SLOT_MAP, S, 0, ref.size)
    off = dev(su.offsets_of(counts)) if ragged else None
    got = smcsd.kv_slot_map(dev(np.array(ctx, np.int32)), dev(table), dev(ref), S, T, page, new_offsets=off,
                            rows=int(sum(counts)) if ragged else None, ws=ws, stream=stream)
    return got, smcsd.check_status(ws)


@pytest.mark.parametrize("G,N,T,page,most", [
    (1, 1, 1, 16, 0), (1, 1, 1, 8, 1), (3, 1, 1, 16, 40), (2, 4, 5, 16, 100), (4, 16, 9, 8, 300), (5, 7, 33, 32, 70),
    (1, 64, 4, 64, 500), (16, 1, 300, 16, 200), (40, 16, 2, 16, 150), (2, 3, 20, 256, 600)])
@pytest.mark.parametrize("ragged", [False, True])
def test_slot_map(smcsd, G, N, T, page, most, ragged):
    rng = np.random.default_rng([G, N, T, page, most])
    S = G * N
    ctx = np.repeat(rng.integers(0, most + 1, G), N).tolist()
    counts = [int(rng.integers(0, T + 1)) for _ in range(S)] if ragged else [T] * S
    counts[0] = max(1, counts[0])
    table, ref = shared_tables(rng, G, N, ctx, T, page, spare=S)
    want = su.slot_map(ctx, counts, table, ref, page)
    got, status = run_slots(smcsd, ctx, counts, T, table, ref, page, ragged)
    assert status == 0
    for k, v in want.items():
        assert np.array_equal(host(got[k]), v), k


def test_slot_map_keeps_pages_that_are_already_there(smcsd):
    # pages taken for drafts that were rejected stay in the table and are used again
    table = np.array([[3, 5, -1, -1]], np.int32)
    ref = np.array([0, 0, 0, 1, 0, 1], np.int32)
    got, status = run_slots(smcsd, [10], [20], 20, table, ref, 16, False)
    assert status == 0
    assert host(got["table_out"]).tolist() == [[3, 5, -1, -1]]
    assert host(got["refcount_out"]).tolist() == ref.tolist()
    assert host(got["slots"]).tolist() == [3 * 16 + i for i in range(10, 16)] + [5 * 16 + i for i in range(14)]


def test_slot_map_of_a_large_pool(smcsd):
    rng = np.random.default_rng(5)
    G, N, page, T = 64, 8, 16, 5
    ctx = np.repeat(rng.integers(0, 400, G), N).tolist()
    table, ref = shared_tables(rng, G, N, ctx, T, page, spare=300001)
    got, status = run_slots(smcsd, ctx, [T] * G * N, T, table, ref, page, False)
    assert status == 0
    for k, v in su.slot_map(ctx, [T] * G * N, table, ref, page).items():
        assert np.array_equal(host(got[k]), v), k


def test_slot_map_errors(smcsd):
    table, ref = np.full((2, 2), -1, np.int32), np.zeros(3, np.int32)

    def status(ctx, counts, t=table, r=ref, ragged=True):
        return run_slots(smcsd, ctx, counts, 64, t, r, 16, ragged)

    assert status([0, 0], [16, 32])[1] == 0
    got, st = status([0, 0], [32, 32])  # four pages, three free
    assert st == smcsd.ERR_PAGES
    assert host(got["table_out"]).tolist() == [[0, 1], [2, -1]]
    assert host(got["slots"])[48:].tolist() == [-1] * 16
    assert status([-1, 0], [1, 1])[1] == smcsd.ERR_RANGE
    assert status([0, 31], [1, 2])[1] == smcsd.ERR_RANGE  # 33 positions of 32
    assert status([0, 0], [1, 1], t=np.array([[7, -1], [-1, -1]], np.int32))[1] == smcsd.ERR_RANGE
    bad = dev(np.array([0, 3, 2], np.int32))
    ws = smcsd.Workspace(smcsd.OP_KV_SLOT_MAP, 2, 0, 3)
    smcsd.kv_slot_map(dev(np.zeros(2, np.int32)), dev(table), dev(ref), 2, 64, 16, new_offsets=bad, rows=3, ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_RANGE


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hkv,D,page,T", [(1, 64, 8, 1), (8, 128, 16, 5), (5, 64, 32, 40), (3, 8, 256, 7)])
def test_append(smcsd, dtype, Hkv, D, page, T):
    rng = np.random.default_rng([Hkv, D, page, T])
    torch.manual_seed(1)
    G, N = 3, 4
    S = G * N
    ctx = np.repeat(rng.integers(0, 90, G), N).tolist()
    counts = [int(rng.integers(1, T + 1)) for _ in range(S)]
    table, ref = shared_tables(rng, G, N, ctx, T, page, spare=S)
    m = su.slot_map(ctx, counts, table, ref, page)
    R, num = sum(counts), ref.size
    m["slots"][R // 2] = -1  # a row that goes nowhere
    kv = torch.randn(R, 3, Hkv, D, device="cuda").to(dtype)
    kc, vc = (torch.randn(num, Hkv, page, D, device="cuda").to(dtype) for _ in range(2))
    wk, wv = kc.clone(), vc.clone()
    for s in range(S):
        if m["copy_src"][s] >= 0:
            part = ctx[s] % page
            for w in (wk, wv):
                w[m["copy_dst"][s], :, :part] = w[m["copy_src"][s], :, :part]
    for r, slot in enumerate(m["slots"]):
        if slot >= 0:
            wk[slot // page, :, slot % page], wv[slot // page, :, slot % page] = kv[r, 1], kv[r, 2]
    ws = smcsd.Workspace(smcsd.OP_KV_APPEND, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    smcsd.kv_append(kv[:, 1], kv[:, 2], dev(m["slots"]), kc, vc, ctx_len=dev(np.array(ctx, np.int32)),
                    copy_src=dev(m["copy_src"]), copy_dst=dev(m["copy_dst"]), ws=ws, stream=stream)
    assert smcsd.check_status(ws, stream) == 0
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_reports_slots_outside_the_cache(smcsd):
    kc = torch.zeros(4, 2, 8, 64, device="cuda")
    vc, new = kc.clone(), torch.ones(2, 2, 64, device="cuda")
    ws = smcsd.Workspace(smcsd.OP_KV_APPEND, 1)
    smcsd.kv_append(new, new, dev(np.array([32, 3], np.int64)), kc, vc, ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_RANGE
    assert int((kc != 0).sum()) == 2 * 64 and bool((kc[0, :, 3] == 1).all())
    one = dev(np.array([1], np.int32))
    smcsd.kv_append(new[:1], new[:1], dev(np.array([3], np.int64)), kc, vc, ctx_len=one,
                    copy_src=dev(np.array([4], np.int32)), copy_dst=one, ws=ws)
    assert smcsd.check_status(ws) == smcsd.ERR_RANGE


@pytest.mark.parametrize("S,T", [(1, 1), (3, 7), (2, 32), (5, 33), (4, 64), (1, 300), (1, 5000)])
@pytest.mark.parametrize("ragged", [False, True])
def test_tree_mask(smcsd, S, T, ragged):
    rng = np.random.default_rng([S, T])
    counts = [int(rng.integers(0, T + 1)) for _ in range(S)] if ragged else [T] * S
    counts[-1] = T
    parents = su.random_parents(counts, rng)
    if T == 5000:
        parents[-2500:] = np.arange(2499, 4999)  # a long chain past the shared part
    ws = smcsd.Workspace(smcsd.OP_TREE_MASK, 1)
    got = smcsd.tree_mask(dev(parents), S, T, node_offsets=dev(su.offsets_of(counts)) if ragged else None, ws=ws)
    assert smcsd.check_status(ws) == 0
    want = su.mask_words(counts, T, su.seen_lists(counts, parents))
    assert np.array_equal(host(got).view(np.uint32), want)


def test_tree_mask_reports_a_parent_that_is_not_before_its_node(smcsd):
    ws = smcsd.Workspace(smcsd.OP_TREE_MASK, 1)
    for bad in ([-1, 1, 0], [-2, 0, 1], [-1, 2, 0]):
        smcsd.tree_mask(dev(np.array(bad, np.int32)), 1, 3, ws=ws)
        assert smcsd.check_status(ws) == smcsd.ERR_RANGE
