"""Attention over long contexts in pages of every size, and groups in which some sequences have no nodes: as
test_attention_long.py, whose cases have pages of 16."""
import numpy as np
import pytest
import torch

import test_attention_long as long
from test_attention_long import BF16, F32, run_and_check

pytestmark = pytest.mark.gpu


@pytest.fixture
def pages(request, monkeypatch):
    monkeypatch.setattr(long, "PAGE", request.param)


@pytest.mark.parametrize("pages", [8, 32, 64, 128, 256], indirect=True)
@pytest.mark.parametrize("dtype,T,g,D", [(BF16, 9, 4, 128), (BF16, 50, 2, 128), (BF16, 70, 4, 128), (BF16, 5, 4, 64), (BF16, 40, 2, 64),
                                         (F32, 4, 4, 128)])
def test_pages_of_every_size(smcsd, pages, dtype, T, g, D):
    # contexts that end anywhere in a page and a tile
    run_and_check(smcsd, T + D, [14801, 14463], [T, T - 1], T, 4 * g, 4, D, dtype, tree=True)


@pytest.mark.parametrize("pages", [8, 64, 256], indirect=True)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,g,D", [(5, 4, 128), (12, 4, 128), (9, 4, 64)])
def test_groups_in_pages_of_every_size(smcsd, pages, dtype, T, g, D):
    # what is shared ends at a page, not at a tile
    N = 4
    ctx = [6000 + 130 * s for s in range(N)] + [3100 + 7 * s for s in range(N)]
    run_and_check(smcsd, T + N, ctx, [T - s % 2 for s in range(2 * N)], T, 4 * g, 4, D, dtype, N=N, shared=2816 + 64)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,g", [(5, 4), (12, 4)])
@pytest.mark.parametrize("counts", [(0, 3, 0, 2), (4, 0, 0, 0), (0, 0, 0, 0, 5, 1, 0, 3), (2, 2, 2, 0, 0, 0, 0, 0)])
def test_groups_with_sequences_that_have_no_nodes(smcsd, dtype, T, g, counts):
    ctx = [2000 + 300 * (s // 4) + s for s in range(len(counts))]
    run_and_check(smcsd, T, ctx, list(counts), T, 4 * g, 4, 128, dtype, N=4, shared=1600)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_sequence_with_nodes_among_many(smcsd, dtype):
    rng = np.random.default_rng(1)
    S = 200
    counts = [0] * S
    counts[131] = 6
    c = run_and_check(smcsd, 1, [int(x) for x in rng.integers(0, 5000, S)], counts, 6, 8, 2, 64, dtype, moving=False)
    assert c.R == 6 and torch.isfinite(c.run(smcsd)[1]).all()
