"""kv_fork and kv_free around the sizes at which one cluster gives way to two launches."""
import numpy as np
import pytest

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,P", [(64, 128), (64, 129), (3, 2731), (8193, 1), (50, 164), (255, 257), (511, 128)])
@pytest.mark.parametrize("more", [0, 1, 5000, 70_000])
def test_tables_and_counts_of_both_forms(smcsd, S, P, more):
    rng = np.random.default_rng(S + P + more)
    num, page = S * P // 2 + more, 16
    table = rng.integers(-1, num, (S, P)).astype(np.int32)
    ref = np.bincount(table[table >= 0], minlength=num).astype(np.int32) + (rng.random(num) < 0.2).astype(np.int32)
    parents = np.where(rng.random(S) < 0.5, np.arange(S), rng.integers(-1, S, S)).astype(np.int32)
    lengths = rng.integers(0, 2 * P * page, S).astype(np.int32)
    ws = smcsd.Workspace(smcsd.OP_KV_FORK, 1)
    got = smcsd.kv_fork(dev(table), dev(ref), dev(parents), page, lengths=dev(lengths), ws=ws)
    want = ou.fork(table, ref, parents, lengths, page)
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    got = smcsd.kv_free(*got, dev(lengths // 2), page, ws=ws)
    want = ou.fork(*want, None, lengths // 2, page)
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    assert smcsd.check_status(ws) == 0
