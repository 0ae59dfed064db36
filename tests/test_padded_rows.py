"""Ragged rows that no sequence has (R padded for a captured graph, offsets that begin above zero), and those of sequences
whose offsets or lengths are refused: they get no slot, and the other operators leave their outputs as they are."""
import numpy as np
import pytest
import torch

import serve_util as su
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


def i32(*a):
    return dev(np.array(a, np.int32))


def slot_map(smcsd, off, rows, ctx=(5, 20, 0), T=8):
    S, P, page = 3, 4, 16
    table = np.full((S, P), -1, np.int32)
    ref = np.zeros(40, np.int32)
    for s in range(S):
        have = (max(ctx[s], 0) + page - 1) // page
        table[s, :have] = 10 * s + np.arange(have)
        ref[table[s, :have]] = 1
    ws = smcsd.Workspace(smcsd.OP_KV_SLOT_MAP, S, 0, ref.size)
    slots = torch.full((rows,), 17, dtype=torch.int64, device="cuda")  # looks like a slot
    got = smcsd.kv_slot_map(i32(*ctx), dev(table), dev(ref), S, T, page, new_offsets=i32(*off), rows=rows, ws=ws, slots=slots)
    assert got["slots"].data_ptr() == slots.data_ptr()
    return smcsd.check_status(ws), host(slots), table, ref


@pytest.mark.parametrize("off,rows", [((0, 2, 5, 6), 6), ((0, 2, 5, 6), 9), ((3, 5, 8, 9), 9), ((2, 4, 4, 4), 2000), ((0, 0, 0, 0), 5)])
def test_rows_of_no_sequence_have_no_slot(smcsd, off, rows):
    status, slots, table, ref = slot_map(smcsd, off, rows)
    assert status == 0
    counts = np.diff(off)
    want = np.full(rows, -1, np.int64)
    want[off[0]:off[-1]] = su.slot_map((5, 20, 0), counts, table, ref, 16)["slots"]
    assert np.array_equal(slots, want)


@pytest.mark.parametrize("off,ctx,refused", [
    ((0, 2, 1, 3), (5, 20, 0), [1]),            # descending
    ((0, 9, 11, 12), (5, 20, 0), [0]),          # more than T
    ((-1, 2, 4, 5), (5, 20, 0), [0]),           # negative
    ((0, 2, 4, 14), (5, 20, 0), [2]),           # past the rows
    ((0, 2, 5, 6), (5, 63, 0), [1]),            # past the table
    ((0, 2, 5, 6), (-3, 20, 0), [0]),           # a negative length
])
def test_rows_of_refused_sequences_have_no_slot(smcsd, off, ctx, refused):
    rows = 13
    status, slots, table, _ = slot_map(smcsd, off, rows, ctx)
    assert status == smcsd.ERR_RANGE
    mine = np.zeros(rows, bool)
    for s in range(3):
        if s not in refused:
            mine[off[s]:off[s + 1]] = True
    assert (slots[~mine] == -1).all() and (slots[mine] >= 0).all()


def test_padding_is_written_nowhere(smcsd):
    # the slots of a padded step go to kv_append as they are
    off, rows = (0, 2, 5, 6), 12
    _, slots, table, _ = slot_map(smcsd, off, rows)
    cache = torch.zeros(40, 1, 16, 64, device="cuda")
    new = torch.ones(rows, 1, 64, device="cuda")
    ws = smcsd.Workspace(smcsd.OP_KV_APPEND, 1)
    smcsd.kv_append(new, new, dev(slots), cache, cache.clone(), ws=ws)
    assert smcsd.check_status(ws) == 0
    assert int(cache.count_nonzero()) == 6 * 64


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off", [(0, 2, 5), (3, 5, 8)])
def test_the_other_operators_leave_padding_as_it_is(smcsd, dtype, off):
    S, T, R, Hq, D, V = 2, 4, 11, 4, 64, 1000
    torch.manual_seed(0)
    rows = slice(off[0], off[-1])
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[rows] = False
    o = i32(*off)
    parents = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    mask = torch.full((R, 1), 77, dtype=torch.int32, device="cuda")
    smcsd.tree_mask(parents, S, T, node_offsets=o, mask=mask)
    assert bool((mask[keep] == 77).all()) and bool((mask[rows] != 77).all())
    q = torch.randn(R, Hq, D, device="cuda").to(dtype)
    k, v = (torch.randn(20, 2, 16, D, device="cuda").to(dtype) for _ in range(2))
    out, lse = torch.full_like(q, 7), torch.full((R, Hq), 7.0, device="cuda")
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    smcsd.tree_attention(q, k, v, table, i32(100, 3), S, T, 0.125, node_offsets=o, mask=mask, out=out, lse=lse)
    assert bool((out[keep] == 7).all()) and bool((lse[keep] == 7).all())
    want, wlse = smcsd.tree_attention(q[rows].contiguous(), k, v, table, i32(100, 3), S, T, 0.125, node_offsets=o - off[0],
                                      mask=mask[rows].contiguous())
    assert torch.equal(out[rows], want) and torch.equal(lse[rows], wlse)
    z = torch.randn(R, V, device="cuda").to(dtype)
    got = smcsd.logits_process(z, S, T, V, node_offsets=o, out=torch.full_like(z, 7))
    assert bool((got[keep] == 7).all()) and torch.equal(got[rows], z[rows])
