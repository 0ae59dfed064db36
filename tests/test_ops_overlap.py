"""Calls that would write memory that they read, or twice what they write, are refused before anything is enqueued, so they are checked
through the C ABI without a GPU."""
import ctypes

from test_serve_args import FAKE, F, I, LL, P, SZ, caller, lib, refused  # noqa: F401

PP, LLP = ctypes.POINTER(P), ctypes.POINTER(LL)


def test_state_reorder_with_another_tensors_memory(lib):  # noqa: F811
    """Three states of 2 * 4 rows of 16, 10 and 3 bytes, and 2 * 4 ancestors of 4 bytes."""
    a, b, c, anc = 1 << 40, 1 << 41, 1 << 42, 1 << 43
    x, y, z = 1 << 44, 1 << 45, 1 << 46
    call = caller(lib.state_reorder, [
        ("src", PP, (P * 3)(a, b, c)), ("dst", PP, (P * 3)(x, y, z)), ("bytes", LLP, (LL * 3)(16, 10, 3)), ("count", I, 3), ("anc", P, P(anc)),
        ("G", I, 2), ("N", I, 4), ("M", I, 4), ("ws", P, FAKE), ("n", SZ, 256), ("stream", P, None)])
    swapped = [(b, a, z), (x, c, b), (c, y, a), (b, c, a)]
    near = [(b + 79, y, z), (b - 127, y, z), (x, a + 127, z), (x, a - 79, z), (x, y, b + 79), (x, y, a - 23)]
    twice = [(x, x, z), (x, x + 127, z), (x, y, x - 23), (x, y, y + 79)]
    ancestors = [(anc, y, z), (x, anc + 31, z), (x, y, anc - 23)]
    refused(call, -1, dst=[(P * 3)(*d) for d in swapped + near + twice + ancestors])
    # one tensor more than a pair, and as many as there may be: the last one's memory is the first one's
    n = 64
    src, dst = [(1 << 40) + 4096 * i for i in range(n)], [(1 << 41) + 4096 * i for i in range(n)]
    dst[-1] = src[0] + 64
    assert call(src=(P * n)(*src), dst=(P * n)(*dst), bytes=(LL * n)(*([16] * n)), count=n) == -1


def test_distill_loss_with_the_lists_memory(lib):  # noqa: F811
    """The gradient's rows of 100 bf16, 220 apart, on the lists, the weights or the losses; the losses on the logits."""
    z, tokens, values, weight, loss, grad = (1 << k for k in range(40, 46))
    call = caller(lib.distill_loss, [
        ("logits", P, P(z)), ("stride", LL, 220), ("dtype", I, 1), ("R", I, 4), ("V", I, 100), ("tokens", P, P(tokens)), ("values", P, P(values)),
        ("K", I, 5), ("T", F, 1.0), ("rest", I, 0), ("weight", P, P(weight)), ("loss", P, P(loss)), ("grad", P, P(grad)), ("gstride", LL, 220),
        ("ws", P, FAKE), ("n", SZ, 256), ("stream", P, None)])
    rows = [0, 440, 3 * 440]  # bytes to the first, second and last row of 200 bytes
    for name, at, size in (("tokens", tokens, 80), ("values", values, 80), ("weight", weight, 16), ("loss", loss, 16)):
        # a row that ends in the list, or begins in it
        refused(call, -1, grad=[P(at - r - 198) for r in rows] + [P(at - r + size - 2) for r in rows])
    refused(call, -1, loss=[P(z + r - 12) for r in rows] + [P(z + r + 196) for r in rows])
    assert call(grad=P(z), loss=P(z + 440 + 196)) == -1  # in place
    assert call(dtype=0, grad=P(loss - 3 * 880 - 396)) == -1 and call(dtype=0, loss=P(z + 880 + 396)) == -1
    for t in (tokens, values, weight):
        assert call(loss=None, grad=P(t)) == -1


def test_kv_compact_with_outputs_that_share_memory(lib):  # noqa: F811
    """4 sequences of 16 pages, 100 counts, lists of 50 moves."""
    at = dict(tout=1 << 42, rout=1 << 43, src=1 << 44, dst=1 << 45, counts=1 << 46)
    size = dict(tout=256, rout=400, src=200, dst=200, counts=8)
    call = caller(lib.kv_compact, [
        ("S", I, 4), ("tin", P, P(1 << 40)), ("tout", P, P(at["tout"])), ("P", I, 16), ("rin", P, P(1 << 41)), ("rout", P, P(at["rout"])), ("num", I, 100),
        ("src", P, P(at["src"])), ("dst", P, P(at["dst"])), ("counts", P, P(at["counts"])), ("ws", P, FAKE), ("n", SZ, 1 << 20), ("stream", P, None)])
    for a in at:
        for b in at:
            if a != b:
                refused(call, -1, **{a: [P(at[b]), P(at[b] + size[b] - 4), P(at[b] - size[a] + 4)]})
