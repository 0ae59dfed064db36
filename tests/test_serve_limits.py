"""Sizes next to the end of 32 bits: rows of node masks and vocabularies whose words or blocks could not be counted are
refused before anything runs. A GPU is not needed."""
import pytest

from test_serve_args import FAKE, I, P, SZ, caller, lib  # noqa: F401

END = 0x7fffffff


def test_node_masks_of_rows_that_cannot_be_counted(lib):  # noqa: F811
    # ragged: T is only a limit, and (T + 31) / 32 words would be negative
    mask = caller(lib.tree_mask, [("parents", P, FAKE), ("off", P, FAKE), ("S", I, 2), ("T", I, 3), ("R", I, 6), ("mask", P, FAKE),
                                  ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    logits = caller(lib.logits_process, [
        ("logits", P, FAKE), ("out", P, FAKE), ("dtype", I, 1), ("R", I, 8), ("V", I, 100), ("S", I, 4), ("T", I, 2), ("off", P, FAKE),
        ("tokens", P, FAKE), ("mask", P, FAKE), ("ht", P, None), ("ho", P, None), ("nh", I, 0), ("rep", P, None), ("pres", P, None),
        ("freq", P, None), ("bt", P, None), ("bv", P, None), ("bo", P, None), ("nb", I, 0), ("allowed", P, None), ("ws", P, FAKE),
        ("n", SZ, 64), ("stream", P, None)])
    slots = caller(lib.kv_slot_map, [
        ("ctx_len", P, FAKE), ("off", P, FAKE), ("S", I, 4), ("T", I, 2), ("R", I, 8), ("tin", P, FAKE), ("tout", P, P(8192)),
        ("P", I, 16), ("page", I, 16), ("rin", P, FAKE), ("rout", P, P(8192)), ("num", I, 100), ("slots", P, FAKE), ("src", P, FAKE),
        ("dst", P, FAKE), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    for call in (mask, logits, slots):
        assert call(T=1 << 20) == -3  # only the workspace is too small
        for T in (END, END - 30, END - 31):
            assert call(T=T) == -1, T
    # the vocabulary's blocks and the grammar mask's words
    for V in (END, END - 30, END - 2000):
        assert logits(V=V) == -1, V
    assert logits(V=1 << 30) == -3


def test_attention_of_rows_that_cannot_be_counted(lib):  # noqa: F811
    size = lib.tree_attention_workspace_size
    for T in (END, END - 31, 1 << 30):
        assert size(1, 1, T, 1, 1, 64) == 0, T
    assert size(1, 1, 1 << 20, 1, 1, 64) > 0


@pytest.mark.parametrize("bad", [0, -1])
def test_no_sizes_below_one(lib, bad):  # noqa: F811
    assert lib.tree_attention_workspace_size(1, 1, bad, 1, 1, 64) == 0
    assert lib.smcsd_workspace_size(7, bad, 0, 10) == 0 and lib.smcsd_workspace_size(7, 1, 0, bad) == 0
