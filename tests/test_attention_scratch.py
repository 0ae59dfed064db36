"""What tree_attention asks for as scratch: pieces for the units that the GPU's blocks can cut, and nothing for the others."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def size():
    from smc_reweight_resample_gb300 import build

    lib = ctypes.CDLL(build.build())
    lib.tree_attention_workspace_size.restype = ctypes.c_size_t
    return lib.tree_attention_workspace_size


FRONT = 1 << 17  # counters, and lists of 64 bytes a sequence come on top


@pytest.mark.parametrize("T,Hq,Hkv,D", [(64, 64, 8, 128), (1, 32, 8, 128), (5, 16, 16, 64), (300, 8, 1, 64)])
@pytest.mark.parametrize("S", [1, 16, 1024, 1025, 5000])
def test_without_groups_two_pieces_a_block(size, S, T, Hq, Hkv, D):
    # up to 160 blocks of up to 256 rows (bf16) or 320 of 16 (float32), each with a unit that is cut at either end
    rows = T * Hq // Hkv
    piece = lambda rb: min(rb, rows) * (4 * D + 8)  # noqa: E731
    most = max(2 * 160 * piece(256), 2 * 320 * piece(16))
    assert size(S, 1, T, Hq, Hkv, D) <= FRONT + 1024 + 64 * S + most


def test_more_sequences_do_not_change_the_order_of_magnitude(size):
    assert size(1025, 1, 64, 64, 8, 128) < 1.1 * size(1024, 1, 64, 64, 8, 128)


def test_with_groups_a_piece_for_each_unit(size):
    # 8 groups of 16 with five nodes, 32 heads on 8: 1024 own units of 20 rows, 64 shared ones of 320 in blocks of 256 at most
    piece = 4 * 128 + 8
    assert size(128, 16, 5, 32, 8, 128) <= FRONT + 64 * 136 + piece * 20 * (1024 + 160) + piece * 256 * (8 * 8 * 3 + 160)
