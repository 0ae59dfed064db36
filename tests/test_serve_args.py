"""Refusals of the operators around the verify: wrong arguments return before anything is enqueued, so
they are checked through the C ABI without a GPU."""
import ctypes

import pytest

P, I, F, SZ, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
FAKE, ODD = P(4096), P(4104)


@pytest.fixture(scope="module")
def lib():
    from smc_reweight_resample_gb300 import build

    lib = ctypes.CDLL(build.build())
    lib.smcsd_workspace_size.restype = lib.tree_attention_workspace_size.restype = SZ
    return lib


def caller(fn, spec):
    """spec: (name, type, default) in order; call(**changed) returns the status."""
    fn.argtypes = [t for _, t, _ in spec]
    fn.restype = I
    names = [n for n, _, _ in spec]

    def call(**k):
        assert set(k) <= set(names), k
        return fn(*[k.get(n, d) for n, _, d in spec])

    return call


def refused(call, code, **cases):
    for name, values in cases.items():
        for v in values:
            assert call(**{name: v}) == code, (name, v)


def test_workspace_sizes(lib):
    assert lib.smcsd_workspace_size(7, 4, 0, 1000) >= 256 + 4 * 1000
    assert lib.smcsd_workspace_size(7, 4, 0, 0) == 0 and lib.smcsd_workspace_size(7, 0, 0, 10) == 0
    for op in (8, 9, 10):
        assert lib.smcsd_workspace_size(op, 1, 0, 1) == 256
    size = lib.tree_attention_workspace_size
    assert size(8, 4, 5, 32, 8, 128) > 0
    for bad in ((0, 1, 5, 32, 8, 128), (8, 3, 5, 32, 8, 128), (8, 1, 0, 32, 8, 128), (8, 1, 5, 30, 8, 128), (8, 1, 5, 32, 0, 128),
                (8, 1, 5, 32, 8, 96), (8, 0, 5, 32, 8, 128)):
        assert size(*bad) == 0, bad


def test_kv_slot_map(lib):
    call = caller(lib.kv_slot_map, [
        ("ctx_len", P, FAKE), ("off", P, None), ("S", I, 4), ("T", I, 2), ("R", I, 8), ("tin", P, FAKE), ("tout", P, P(8192)),
        ("P", I, 16), ("page", I, 16), ("rin", P, FAKE), ("rout", P, P(8192)), ("num", I, 100), ("slots", P, FAKE), ("src", P, FAKE),
        ("dst", P, FAKE), ("ws", P, FAKE), ("n", SZ, 256), ("stream", P, None)])
    assert call() == -3
    assert call(n=1 << 20, ws=P(4100)) == -3
    refused(call, -1, ctx_len=[None], tin=[None, P(8192)], tout=[None], rin=[None], rout=[None, FAKE], slots=[None], src=[None],
            dst=[None], S=[0, -1, 3], T=[0, 3], R=[0, 7], P=[0, 1 << 28], page=[0, 4, 12, 512, -16], num=[0], ws=[None])


def test_kv_append(lib):
    call = caller(lib.kv_append, [
        ("k", P, FAKE), ("v", P, FAKE), ("dtype", I, 1), ("R", I, 4), ("Hkv", I, 2), ("D", I, 64), ("stride", LL, 128),
        ("slots", P, FAKE), ("src", P, FAKE), ("dst", P, FAKE), ("ctx", P, FAKE), ("S", I, 2), ("kc", P, FAKE), ("vc", P, FAKE),
        ("page", I, 16), ("num", I, 10), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -2, dtype=[2, -1])
    refused(call, -1, k=[None, ODD], v=[None, ODD], slots=[None], kc=[None, ODD], vc=[None, ODD], src=[None], dst=[None], ctx=[None],
            S=[0], R=[0], Hkv=[0], D=[0, 60, 100], stride=[127, 132], page=[24], num=[0], ws=[None])


def test_tree_mask(lib):
    call = caller(lib.tree_mask, [("parents", P, FAKE), ("off", P, None), ("S", I, 2), ("T", I, 3), ("R", I, 6), ("mask", P, FAKE),
                                  ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -1, parents=[None], mask=[None], S=[0], T=[0], R=[5, 0], ws=[None])


def test_tree_attention(lib):
    call = caller(lib.tree_attention, [
        ("q", P, FAKE), ("q_stride", LL, 512), ("kc", P, FAKE), ("vc", P, FAKE), ("dtype", I, 1), ("num", I, 100), ("page", I, 16),
        ("table", P, FAKE), ("P", I, 8), ("ctx", P, FAKE), ("off", P, None), ("S", I, 4), ("N", I, 2), ("T", I, 2), ("R", I, 8),
        ("mask", P, None), ("Hq", I, 8), ("Hkv", I, 2), ("D", I, 64), ("scale", F, 0.125), ("out", P, FAKE), ("lse", P, None),
        ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -2, dtype=[2, 7])
    refused(call, -1, q=[None, ODD], kc=[None, ODD], vc=[None, ODD], table=[None], ctx=[None], out=[None, ODD], q_stride=[511, 516],
            num=[0], page=[4, 48, 512], P=[0, 1 << 27], S=[0, 3], N=[0, 3], T=[0, 3], R=[0, 9], Hq=[0, 7], Hkv=[0, 3], D=[32, 96, 0],
            scale=[float("nan"), float("inf")], ws=[None])


def test_logits_process(lib):
    call = caller(lib.logits_process, [
        ("logits", P, FAKE), ("out", P, FAKE), ("dtype", I, 1), ("R", I, 8), ("V", I, 100), ("S", I, 4), ("T", I, 2), ("off", P, None),
        ("tokens", P, FAKE), ("mask", P, FAKE), ("ht", P, FAKE), ("ho", P, FAKE), ("nh", I, 5), ("rep", P, None), ("pres", P, None),
        ("freq", P, None), ("bt", P, FAKE), ("bv", P, FAKE), ("bo", P, FAKE), ("nb", I, 5), ("allowed", P, None), ("ws", P, FAKE),
        ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -2, dtype=[2])
    refused(call, -1, logits=[None], out=[None], R=[0, 7], V=[0], S=[0], T=[0, 3], tokens=[None], ht=[None], ho=[None], nh=[-1],
            bt=[None], bv=[None], bo=[None], nb=[-1], ws=[None])
    assert call(S=70000, R=140000) == -1


def test_the_python_calls_refuse_wrong_tensors():
    import torch

    from smc_reweight_resample_gb300 import _binding as B

    class Ws:
        ptr, nbytes = 4096, 1 << 20

    i32 = torch.zeros(4, dtype=torch.int32)
    q, cache = torch.zeros(2, 4, 64), torch.zeros(3, 2, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        B.tree_mask(i32, 1, 4, ws=Ws)
    with pytest.raises(TypeError):
        B._native().tree_mask("parents", 1, 4, None, None, 1, 1, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.tree_attention(q, cache, cache, i32.view(1, 4), i32, 1, 2, 1.0, ws=Ws)
    with pytest.raises(TypeError, match="one type"):
        B.tree_attention(q, cache, cache.bfloat16(), i32.view(1, 4), i32, 1, 2, 1.0, ws=Ws)
    with pytest.raises(ValueError, match="alike"):
        B.tree_attention(q, cache, cache[:2], i32.view(1, 4), i32, 1, 2, 1.0, ws=Ws)
    with pytest.raises(ValueError, match="pages_per_seq"):
        B.kv_slot_map(i32, i32, i32, 4, 1, 16, ws=Ws)
    with pytest.raises(ValueError, match="rows"):
        B.kv_slot_map(i32, i32.view(1, 4), i32, 1, 1, 16, new_offsets=i32, ws=Ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.logits_process(q, 1, 2, 128, ws=Ws)
    with pytest.raises(ValueError, match="node_tokens"):
        B.logits_process(torch.zeros(8, 10), 8, 1, 10, node_tokens=i32, ws=Ws)
