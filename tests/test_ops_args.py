"""Refusals of beam selection, the pages' housekeeping and the distillation loss: wrong arguments return before anything is
enqueued, so they are checked through the C ABI without a GPU."""
import ctypes

import pytest

from test_serve_args import FAKE, F, I, LL, ODD, P, SZ, caller, lib, refused  # noqa: F401

END = 0x7fffffff
FAR = P(1 << 40)


def test_workspace_sizes(lib):  # noqa: F811
    size = lib.smcsd_workspace_size
    for op in (12, 13, 15):
        assert size(op, 1, 0, 1) == 256 and size(op, 0, 0, 1) == 0
    assert size(11, 128, 0, 128256) >= 128 * 126 * (8 + 32 + 8)
    assert size(11, 1, 0, 0) == 0 and size(11, 0, 0, 5) == 0 and size(11, 1, 0, END) == 0
    assert size(14, 1, 0, 1000) >= 4000 and size(14, 1, 0, 0) == 0
    assert size(16, 1, 0, 10) == 0


def test_beam_select(lib):  # noqa: F811
    call = caller(lib.beam_select, [
        ("logits", P, FAKE), ("stride", LL, 100), ("dtype", I, 1), ("G", I, 4), ("N", I, 2), ("V", I, 100), ("M", I, 3), ("T", F, 1.0),
        ("scores", P, FAR), ("finished", P, FAR), ("pad", I, 0), ("eos", I, -1), ("tokens", P, FAKE), ("anc", P, FAKE), ("out", P, FAKE),
        ("over", P, FAKE), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    assert call(n=1 << 24, ws=P(4100)) == -3
    refused(call, -2, dtype=[2, -1])
    refused(call, -1, logits=[None, P(4097)], stride=[99, 0, -100], G=[0, -1, 1 << 30], N=[0, 257, -2], V=[0, -5, END, END - 100], M=[0, 257, -1],
            T=[0.0, -1.0, float("nan"), float("inf"), 1e-45], tokens=[None], anc=[None], out=[None, FAR], over=[FAR], ws=[None])
    assert call(scores=None, finished=None, over=None) == -3
    assert call(V=1 << 30, N=256, stride=1 << 30) == -1  # a group's chunks could not be counted


def test_state_reorder(lib):  # noqa: F811
    PP, LLP = ctypes.POINTER(P), ctypes.POINTER(LL)

    def ptrs(*a):
        return (P * len(a))(*a)

    def sizes(*a):
        return (LL * len(a))(*a)
    call = caller(lib.state_reorder, [
        ("src", PP, ptrs(4096, 8192)), ("dst", PP, ptrs(1 << 40, 1 << 41)), ("bytes", LLP, sizes(16, 10)), ("count", I, 2), ("anc", P, FAKE), ("G", I, 2),
        ("N", I, 4), ("M", I, 4), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -1, src=[None], dst=[None], bytes=[None], count=[0, 65, -1], anc=[None], G=[0, 1 << 30], N=[0], M=[0], ws=[None])
    # what is looked at with a workspace of the right size: null pointers, sizes, and memory that is read and written
    for bad in (dict(src=ptrs(4096, None)), dict(dst=ptrs(None, 1 << 41)), dict(bytes=sizes(16, 0)), dict(bytes=sizes(-4, 10)),
                dict(bytes=sizes(1 << 62, 10)), dict(dst=ptrs(4096, 1 << 41)), dict(dst=ptrs(1 << 40, 8192 + 79)), dict(dst=ptrs(1 << 40, 8192 - 79))):
        assert call(n=256, **bad) == -1, bad


@pytest.mark.parametrize("name", ["kv_fork", "kv_free"])
def test_kv_fork_and_free(lib, name):  # noqa: F811
    call = caller(getattr(lib, name), ([("parents", P, FAKE)] if name == "kv_fork" else []) + [
        ("lengths", P, FAKE), ("S", I, 4), ("tin", P, FAKE), ("tout", P, P(8192)), ("P", I, 16), ("page", I, 16), ("rin", P, FAKE),
        ("rout", P, P(8192)), ("num", I, 100), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -1, S=[0, -1], tin=[None, P(8192)], tout=[None], P=[0, 1 << 28], page=[0, 4, 12, 512, -16], rin=[None], rout=[None, FAKE], num=[0],
            ws=[None])
    if name == "kv_fork":
        refused(call, -1, parents=[None])
        assert call(lengths=None) == -3
    else:
        refused(call, -1, lengths=[None])


def test_kv_compact(lib):  # noqa: F811
    call = caller(lib.kv_compact, [
        ("S", I, 4), ("tin", P, FAKE), ("tout", P, P(8192)), ("P", I, 16), ("rin", P, FAKE), ("rout", P, P(8192)), ("num", I, 100), ("src", P, FAKE),
        ("dst", P, P(8192)), ("counts", P, FAKE), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -1, S=[0], tin=[None, P(8192)], tout=[None], P=[0], rin=[None], rout=[None, FAKE], num=[0, -4, END], src=[None, P(8192)],
            dst=[None], counts=[None], ws=[None])
    assert call(num=1, src=None, dst=None) == -3


def test_kv_copy_pages(lib):  # noqa: F811
    PP = ctypes.POINTER(P)
    caches = (P * 3)(4096, 8192, 12288)
    call = caller(lib.kv_copy_pages, [
        ("caches", PP, caches), ("count_caches", I, 3), ("bytes", LL, 4096), ("num", I, 10), ("src", P, FAKE), ("dst", P, FAKE), ("n_moves", I, 4),
        ("count", P, None), ("ws", P, FAKE), ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -1, caches=[None], count_caches=[0, 257, -1], bytes=[0, 24, -16, 1 << 33], num=[0], src=[None], dst=[None], n_moves=[0, -1], ws=[None])
    for bad in ((P * 3)(4096, None, 8192), (P * 3)(4096, 4104, 8192)):
        assert call(caches=bad, n=256) == -1


def test_distill_loss(lib):  # noqa: F811
    call = caller(lib.distill_loss, [
        ("logits", P, FAKE), ("stride", LL, 100), ("dtype", I, 1), ("R", I, 4), ("V", I, 100), ("tokens", P, FAKE), ("values", P, FAKE), ("K", I, 5),
        ("T", F, 1.0), ("rest", I, 0), ("weight", P, None), ("loss", P, FAKE), ("grad", P, FAR), ("gstride", LL, 100), ("ws", P, FAKE),
        ("n", SZ, 64), ("stream", P, None)])
    assert call() == -3
    refused(call, -2, dtype=[2, 9])
    refused(call, -1, logits=[None, P(4097)], stride=[99, -100], R=[0, -1, END], V=[0, -1, 819185], tokens=[None], values=[None], K=[0, 257],
            T=[0.0, -2.0, float("nan"), float("inf"), 1e-45], rest=[2, -1], grad=[P((1 << 40) + 1)], gstride=[99, 0], ws=[None])
    assert call(loss=None, grad=None) == -1
    assert call(loss=None) == -3 and call(grad=None, gstride=0) == -3
    assert call(grad=FAKE, gstride=128) == -1 and call(grad=FAKE, gstride=100) == -3  # in place: one stride
    for dtype, most in ((1, 819184), (0, 409592)):
        assert call(dtype=dtype, V=most, stride=most, gstride=most) == -3
        assert call(dtype=dtype, V=most + 1, stride=most + 1, gstride=most + 1) == -1


def test_outputs_that_overlap_inputs(lib):  # noqa: F811
    """Every call here is refused: what is written would meet what is read."""
    beam = caller(lib.beam_select, [
        ("logits", P, FAKE), ("stride", LL, 100), ("dtype", I, 1), ("G", I, 4), ("N", I, 2), ("V", I, 100), ("M", I, 3), ("T", F, 1.0),
        ("scores", P, FAR), ("finished", P, P(1 << 41)), ("pad", I, 0), ("eos", I, -1), ("tokens", P, FAKE), ("anc", P, FAKE), ("out", P, FAKE),
        ("over", P, FAKE), ("ws", P, FAKE), ("n", SZ, 1 << 24), ("stream", P, None)])
    refused(beam, -1, **{out: [P((1 << 40) + 28), P((1 << 40) - 44), P((1 << 41) + 4)] for out in ("tokens", "anc", "out", "over")})
    for name in ("kv_fork", "kv_free"):
        fork = caller(getattr(lib, name), ([("parents", P, FAKE)] if name == "kv_fork" else []) + [
            ("lengths", P, FAKE), ("S", I, 4), ("tin", P, FAR), ("tout", P, P(8192)), ("P", I, 16), ("page", I, 16), ("rin", P, P(1 << 41)),
            ("rout", P, P(1 << 42)), ("num", I, 100), ("ws", P, FAKE), ("n", SZ, 256), ("stream", P, None)])
        refused(fork, -1, tout=[P((1 << 40) + 252), P((1 << 40) - 252), P((1 << 41) + 4), P(4096 + 12)], rout=[P((1 << 40) - 396), P((1 << 41) + 396), FAKE])
    compact = caller(lib.kv_compact, [
        ("S", I, 4), ("tin", P, FAR), ("tout", P, P(8192)), ("P", I, 16), ("rin", P, P(1 << 41)), ("rout", P, P(1 << 42)), ("num", I, 100),
        ("src", P, P(1 << 43)), ("dst", P, P(1 << 44)), ("counts", P, P(1 << 45)), ("ws", P, FAKE), ("n", SZ, 1 << 20), ("stream", P, None)])
    near = [P((1 << 40) + 252), P((1 << 41) + 396)]
    refused(compact, -1, tout=near, rout=near, src=near, dst=near, counts=near)
    distill = caller(lib.distill_loss, [
        ("logits", P, FAR), ("stride", LL, 220), ("dtype", I, 1), ("R", I, 4), ("V", I, 100), ("tokens", P, P(1 << 41)), ("values", P, P(1 << 42)),
        ("K", I, 5), ("T", F, 1.0), ("rest", I, 0), ("weight", P, P(1 << 43)), ("loss", P, FAKE), ("grad", P, P(1 << 44)), ("gstride", LL, 220),
        ("ws", P, FAKE), ("n", SZ, 256), ("stream", P, None)])
    refused(distill, -1, grad=[P((1 << 40) + d) for d in (2, 198, -2, -198, 440 + 198, 242, 1320 + 198, -1320 - 198)],
            loss=[P((1 << 41) + 76), P((1 << 42) - 12), P((1 << 43) + 4)])
    assert distill(grad=P((1 << 40) + 200), gstride=440) == -1  # between the logits' rows, but not all of them


def test_the_python_calls_refuse_wrong_tensors():
    import torch

    from smc_reweight_resample_gb300 import _binding as B

    class Ws:
        ptr, nbytes = 4096, 1 << 20

    i32 = torch.zeros(4, dtype=torch.int32)
    z = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="CUDA"):
        B.beam_select(z, 2, 2, 10, 3, ws=Ws)
    with pytest.raises(ValueError, match="rows"):
        B.beam_select(z, 2, 3, 10, 3, ws=Ws)
    with pytest.raises(ValueError, match="rows of V"):
        B.beam_select(z, 2, 2, 11, 3, ws=Ws)
    with pytest.raises(ValueError, match="rows of V"):
        B.beam_select(z.t(), 5, 2, 4, 3, ws=Ws)
    with pytest.raises(ValueError, match="rows of V"):
        B.beam_select(z[:1].expand(4, 10), 2, 2, 10, 3, ws=Ws)
    with pytest.raises(TypeError, match="bfloat16"):
        B.beam_select(z.half(), 2, 2, 10, 3, ws=Ws)
    with pytest.raises(ValueError, match="scores"):
        B.beam_select(z, 2, 2, 10, 3, scores=torch.zeros(3), ws=Ws)
    with pytest.raises(ValueError, match="positive"):
        B.beam_select(z, 0, 2, 10, 3, ws=Ws)
    with pytest.raises(TypeError, match="list"):
        B.state_reorder(z, i32, 2, 2, ws=Ws)
    with pytest.raises(ValueError, match="1 to 64"):
        B.state_reorder([], i32, 2, 2, ws=Ws)
    with pytest.raises(ValueError, match="1 to 64"):
        B.state_reorder([z] * 65, i32, 2, 2, ws=Ws)
    with pytest.raises(TypeError, match="tensor"):
        B.state_reorder([1], i32, 2, 2, ws=Ws)
    with pytest.raises(ValueError, match="ancestors"):
        B.state_reorder([z], i32, 2, 3, ws=Ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.state_reorder([z], i32, 2, 2, ws=Ws)
    with pytest.raises(ValueError, match="pages_per_seq"):
        B.kv_fork(i32, i32, i32, 16, ws=Ws)
    with pytest.raises(ValueError, match="parents"):
        B.kv_fork(i32.view(4, 1), i32, i32[:3], 16, ws=Ws)
    with pytest.raises(ValueError, match="lengths"):
        B.kv_free(i32.view(4, 1), i32, i32[:3], 16, ws=Ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_compact(i32.view(2, 2), i32, ws=Ws)
    with pytest.raises(ValueError, match="alike"):
        B.kv_copy_pages([z], i32, i32[:2], ws=Ws)
    with pytest.raises(TypeError, match="list"):
        B.kv_copy_pages(z, i32, i32, ws=Ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_copy_pages([z], i32, i32, ws=Ws)
    with pytest.raises(ValueError, match="top_tokens"):
        B.distill_loss(z, i32.view(2, 2), torch.zeros(2, 2), 10, ws=Ws)
    with pytest.raises(ValueError, match="top_tokens"):
        B.distill_loss(z, i32.view(4, 1), torch.zeros(4, 2), 10, ws=Ws)
    with pytest.raises(ValueError, match="weight"):
        B.distill_loss(z, i32.view(4, 1), torch.zeros(4, 1), 10, weight=torch.zeros(3), ws=Ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.distill_loss(z, i32.view(4, 1), torch.zeros(4, 1), 10, ws=Ws)
