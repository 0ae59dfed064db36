"""Beam selection, the pages' housekeeping and distillation in the examples' runs, on other streams, in shared workspaces."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import ops_util as ou
from gpu_util import dev, host

pytestmark = pytest.mark.gpu


def load_example(name):
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", name + ".py")
    spec = importlib.util.spec_from_file_location(name, path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# ------------------------------------------------------------------------------------------------
# a beam search against one that starts each hypothesis from its tokens, in float64
# ------------------------------------------------------------------------------------------------

def reference_logits(search, tokens):
    """Logits after `tokens`, from the model's tables in float64."""
    Hq, Hkv, D = search.Hq, search.Hkv, search.D
    qkv = search.qkv.double()[torch.tensor(tokens, device="cuda")]
    q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
    q, k, v = q[-1].view(Hq, D), k.view(-1, Hkv, D).repeat_interleave(Hq // Hkv, 1), v.view(-1, Hkv, D).repeat_interleave(Hq // Hkv, 1)
    p = torch.softmax(torch.einsum("hd,xhd->hx", q, k) * D ** -0.5, 1)
    o = torch.einsum("hx,xhd->hd", p, v).flatten()
    return ou.as_float64((search.embed.double()[tokens[-1]] + o @ search.w_out.double()) @ search.head.double())


@pytest.mark.parametrize("G,N,page,prompt,eos", [(3, 4, 16, (40, 17, 64), 5), (2, 8, 8, (9, 30), -1), (1, 1, 16, (33,), -1), (4, 3, 16, (1, 2, 16, 31), 7)])
def test_beam_search(smcsd, G, N, page, prompt, eos):
    search = load_example("beam_search").Search(G=G, N=N, page=page, pages_per_seq=192 // page, prompt=prompt, eos=eos, seed=G + N)
    start = host(search.ctx)[::N].copy()
    beams = [[(host(search.tokens)[g * N, :start[g] + 1].tolist(), 0.0, False)] for g in range(G)]
    for step in range(12):
        search.step()
        for g in range(G):
            cand = []
            for i, (toks, score, over) in enumerate(beams[g]):
                if over:
                    cand.append((score, i, -1))
                    continue
                z = reference_logits(search, toks)
                logp = z - (z.max() + np.log(np.exp(z - z.max()).sum()))
                cand += [(score + x, i, v) for v, x in enumerate(logp)]
            cand.sort(key=lambda c: (-c[0], c[1], c[2]))
            gaps = [a[0] - b[0] for a, b in zip(cand[:N], cand[1:N + 1])]
            assert min(gaps) > 1e-4, "the case's order is not certain in float32"
            beams[g] = [(beams[g][i][0] + [eos if v < 0 else v], s, v < 0 or (eos >= 0 and v == eos)) for s, i, v in cand[:N]]
        tokens, scores, ctx = host(search.tokens), host(search.scores), host(search.ctx)
        for g in range(G):
            for n, (toks, score, over) in enumerate(beams[g]):
                s = g * N + n
                assert tokens[s, :ctx[s] + 1].tolist() == toks
                # float32 logits of two products of 128 and 256 and scores of up to 12 steps
                assert abs(scores[s] - score) < 1e-3 and bool(host(search.finished)[s]) == over
    search.check()
    # the counts are those of the tables, and every beam's pages hold its own tokens' keys and values
    for release in ([], [0], list(range(G))):
        if release:
            used = int(search.release(release))
            search.check()
            assert used == int((search.refcount > 0).sum()) and not bool((search.refcount[used:] > 0).any())
        table, ref = host(search.table), host(search.refcount)
        assert np.array_equal(ref, np.bincount(table[table >= 0].ravel(), minlength=ref.size))
        for s in range(G * N):
            n = int(search.ctx[s])
            pages = search.table[s, :(n + page - 1) // page].long()
            if s // N in release:
                assert (table[s] == -1).all()
                continue
            kv = search.qkv[search.tokens[s, :n].long()][:, search.Hq * search.D:].unflatten(1, (2, search.Hkv, search.D))
            for i, cache in enumerate(search.caches):
                assert torch.equal(cache[pages].permute(0, 2, 1, 3).flatten(0, 1)[:n], kv[:, i])


def test_beam_search_goes_on_after_compaction(smcsd):
    example = load_example("beam_search")
    a, b = example.Search(seed=4), example.Search(seed=4)
    for step in range(8):
        if step in (2, 5):
            b.release([])  # nothing is let go; pages move
        a.step(), b.step()
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.scores, b.scores)
    b.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_distilled_draft(smcsd, dtype):
    draft = load_example("distill_draft").Draft(R=48, V=1500, width=64, K=20, temperature=1.5, seed=1, dtype=dtype)
    hidden = draft.hidden()
    tokens, values = draft.teacher(hidden)
    weight = torch.rand(48, device="cuda")
    loss, grad = draft.gradient(hidden, tokens, values, weight)
    draft.check()
    z = ou.as_float64(hidden @ draft.head)
    want, dwant, scale, parts = ou.distill(z, host(tokens), host(values), 1500, 1.5, True, host(weight))
    assert (np.abs(ou.as_float64(loss) - want) <= 128 * 2.0 ** -24 * scale).all()
    h = ou.as_float64(hidden)
    # each element of dlogits: the kernel's error and its rounding; the product adds 48 of them in float32 (bf16: rounded once more)
    eps = torch.finfo(dtype).eps / 2
    one = 640 * 2.0 ** -24 * parts + eps * np.abs(dwant)
    bound = np.abs(h).T @ (one + 48 * 2.0 ** -24 * (np.abs(dwant) + one))
    exact = h.T @ dwant
    got = ou.as_float64(grad)
    assert (np.abs(got - exact) <= bound + eps * (np.abs(exact) + bound) + 1e-12).all()
    for _ in range(3):  # and it runs
        draft.step()
    draft.check()


# ------------------------------------------------------------------------------------------------
# streams and workspaces
# ------------------------------------------------------------------------------------------------

SPIN = 60_000_000  # clocks: about 30 ms


def operators(smcsd):
    """name: (call(inputs, **how), inputs, workspace)"""
    torch.manual_seed(0)
    rng = np.random.default_rng(0)
    table = rng.permutation(60).astype(np.int32).reshape(6, 10)
    ref = np.concatenate([np.ones(60), np.zeros(40)]).astype(np.int32)
    z = torch.randn(6, 5000, device="cuda")
    top, at = torch.log_softmax(z + torch.randn_like(z), 1).topk(10, 1)
    cache = torch.randn(100, 2, 8, 64, device="cuda")
    return {
        "beam_select": (lambda i, **how: smcsd.beam_select(i[0], 2, 3, 5000, 4, scores=i[1], **how), (z, torch.randn(6, device="cuda")),
                        lambda: smcsd.Workspace(smcsd.OP_BEAM_SELECT, 6, 0, 5000)),
        "top": (lambda i, **how: smcsd.beam_select(i[0], 6, 1, 5000, 9, **how), (z,), lambda: smcsd.Workspace(smcsd.OP_BEAM_SELECT, 6, 0, 5000)),
        "state_reorder": (lambda i, **how: tuple(smcsd.state_reorder(list(i[1:]), i[0], 2, 3, **how)),
                          (dev(np.array([2, 0, 0, 1, 1, 2], np.int32)), z, torch.randn(6, 7, device="cuda")),
                          lambda: smcsd.Workspace(smcsd.OP_STATE_REORDER, 1)),
        "kv_fork": (lambda i, **how: smcsd.kv_fork(i[0], i[1], i[2], 16, **how), (dev(table), dev(ref), dev(np.array([3, 1, -1, 3, 0, 0], np.int32))),
                    lambda: smcsd.Workspace(smcsd.OP_KV_FORK, 1)),
        "kv_free": (lambda i, **how: smcsd.kv_free(i[0], i[1], i[2], 16, **how), (dev(table), dev(ref), dev(np.array([0, 16, 17, 500, 3, 159], np.int32))),
                    lambda: smcsd.Workspace(smcsd.OP_KV_FORK, 1)),
        "kv_compact": (lambda i, **how: smcsd.kv_compact(i[0], i[1], **how), (dev(table), dev(np.roll(ref, 25) * 1)),
                       lambda: smcsd.Workspace(smcsd.OP_KV_COMPACT, 1, 0, 100)),
        "kv_copy_pages": (lambda i, **how: tuple(smcsd.kv_copy_pages([i[0]], i[1], i[2], **how)),
                          (cache, dev(np.array([90, 91, 92], np.int32)), dev(np.array([1, 2, 5], np.int32))), lambda: smcsd.Workspace(smcsd.OP_KV_FORK, 1)),
        "distill_loss": (lambda i, **how: smcsd.distill_loss(i[0], i[1], i[2], 5000, rest=True, **how), (z, at.int(), top),
                         lambda: smcsd.Workspace(smcsd.OP_DISTILL_LOSS, 1)),
    }


NAMES = ["beam_select", "top", "state_reorder", "kv_fork", "kv_free", "kv_compact", "kv_copy_pages", "distill_loss"]


def tensors(got):
    return [t for t in (got.values() if isinstance(got, dict) else got) if t is not None]


def case(smcsd, name):
    call, inputs, ws = operators(smcsd)[name]
    table_in_range = name != "kv_compact"
    if not table_in_range:  # the tables' pages are those in use
        ref = host(inputs[1])
        used = np.nonzero(ref)[0].astype(np.int32)
        inputs = (dev(used.reshape(6, 10)), inputs[1])
    want = [t.clone() for t in tensors(call(tuple(t.clone() for t in inputs)))]
    torch.cuda.synchronize()
    return call, inputs, ws, want


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream_with_work_pending_and_inputs_released(smcsd, name):
    call, inputs, _, want = case(smcsd, name)
    side = torch.cuda.Stream()
    # blocks that hold no zeros, whose last use on the caller's stream is still to come
    given = tuple(t.clone() for t in inputs)
    torch.cuda.synchronize()
    torch.cuda._sleep(SPIN)
    for n in (16, 64, 256, 1024, 4096, 20_000, 80_000, 600_000):
        for _ in range(3):
            torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
    got = call(given, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(tensors(got), want):
        assert torch.equal(a, b)
    # and the other stream held up while the caller lets go of the inputs
    given = tuple(t.clone() for t in inputs)
    shapes = [(t.shape, t.dtype) for t in given]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SPIN)
    got = call(given, stream=side)
    del given
    for shape, dtype in shapes:
        for _ in range(4):
            torch.zeros(shape, dtype=dtype, device="cuda")
    torch.cuda.synchronize()
    for a, b in zip(tensors(got), want):
        assert torch.equal(a, b)


def test_one_workspace_for_all_in_turn(smcsd):
    cases = [case(smcsd, name) for name in NAMES]
    sizes = [ws().nbytes for _, _, ws, _ in cases] + [smcsd.workspace_size(smcsd.OP_KV_SLOT_MAP, 4, 0, 3000)]
    one = object.__new__(smcsd.Workspace)
    one._allocate(max(sizes), None)
    junk = dev(np.zeros(3000, np.int32))
    order = list(range(len(NAMES))) * 2 + [j for k in range(len(NAMES)) for j in (k, 0, k)]
    for i in order:
        call, inputs, _, want = cases[i]
        got = call(tuple(t.clone() for t in inputs), ws=one)
        assert smcsd.check_status(one) == 0
        for a, b in zip(tensors(got), want):
            assert torch.equal(a, b), NAMES[i]
        front = one.buf[one.ptr - one.buf.data_ptr():][256:17408]
        assert int(front.count_nonzero()) == 0, NAMES[i]
        smcsd.kv_slot_map(dev(np.full(4, 3, np.int32)), dev(np.full((4, 3), -1, np.int32)), junk, 4, 2, 16, ws=one)
        assert smcsd.check_status(one) == 0


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_with_one_workspace(smcsd, name):
    call, inputs, ws, want = case(smcsd, name)
    shared = ws()
    given = tuple(t.clone() for t in inputs)
    call(given, ws=shared)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(tensors(call(given, ws=shared)))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert smcsd.check_status(shared) == 0
    for got in outs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------------
# kernels whose launch goes on beside the one before them: each call's input is the output of the one before
# ------------------------------------------------------------------------------------------------

def chain(smcsd, st, wait, between):
    """Selection, states, tables, forks, freeing, compaction and copies, each from what the one before wrote."""
    z, states, table, ref, cache = (st[k] for k in ("z", "states", "table", "ref", "cache"))
    G, N, V, P, num = 3, 4, 700, 40, 900
    S = G * N
    ws = st["ws"]
    states, cache, scores = states.clone(), cache.clone(), torch.zeros(S, device="cuda")
    for step in range(6):
        best = smcsd.beam_select(z[step], G, N, V, N, scores=scores, ws=ws["beam"])
        wait()
        scores = best["scores"]
        states, = smcsd.state_reorder([states], best["ancestors"], G, N, ws=ws["state"])
        wait()
        table, ref = smcsd.kv_pagetable_remap(best["ancestors"], None, G, N, table, P, num, ws=ws["remap"])
        wait()
        states2 = between(states)
        parents = (best["tokens"] % S).to(torch.int32)
        wait()
        table, ref = smcsd.kv_fork(table, ref, parents, 16, ws=ws["fork"])
        wait()
        lengths = states2[:, 0].abs().to(torch.int32) % (P * 16)
        table, ref = smcsd.kv_free(table, ref, lengths, 16, ws=ws["fork"])
        wait()
        moved = smcsd.kv_compact(table, ref, ws=ws["compact"])
        wait()
        table, ref = moved["table_out"], moved["refcount_out"]
        smcsd.kv_copy_pages([cache], moved["src"], moved["dst"], count=moved["counts"], ws=ws["fork"])
        wait()
        states, = smcsd.state_reorder([states2], best["ancestors"], G, N, ws=ws["state"])
        wait()
    return scores, states, table, ref, cache


@pytest.mark.parametrize("how", ["stream", "graph", "copies between", "two streams", "graph of two streams"])
def test_a_chain_without_a_wait_is_the_one_with_waits(smcsd, how):
    G, N, V, P, num = 3, 4, 700, 40, 900
    S = G * N
    rng = np.random.default_rng(5)
    gen = torch.Generator("cuda").manual_seed(5)
    z = torch.randn(6, S, V, device="cuda", generator=gen) * 3
    states = torch.randint(-20_000, 20_000, (S, 333), device="cuda", generator=gen, dtype=torch.int32)
    table = np.where(rng.random((S, P)) < 0.8, rng.integers(0, num, (S, P)), -1).astype(np.int32)
    ref = np.bincount(table[table >= 0], minlength=num).astype(np.int32)
    cache = torch.randn(num, 64, device="cuda", generator=gen)
    ws = dict(beam=smcsd.Workspace(smcsd.OP_BEAM_SELECT, S, 0, V), state=smcsd.Workspace(smcsd.OP_STATE_REORDER, 1),
              remap=smcsd.Workspace(smcsd.OP_PAGETABLE_REMAP, G), fork=smcsd.Workspace(smcsd.OP_KV_FORK, 1),
              compact=smcsd.Workspace(smcsd.OP_KV_COMPACT, 1, 0, num))
    st = dict(z=z, states=states, table=dev(table), ref=dev(ref), cache=cache, ws=ws)
    side = torch.cuda.Stream()

    def copied(x):
        y = torch.zeros_like(x)
        y.copy_(x)
        return y

    def aside(x):  # by way of another stream
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            y = torch.empty_like(x)
            y.copy_(x)
        here.wait_stream(side)
        y.record_stream(here)
        return y

    want = chain(smcsd, st, torch.cuda.synchronize, lambda x: x)
    torch.cuda.synchronize()
    between = {"copies between": copied, "two streams": aside, "graph of two streams": aside}.get(how, lambda x: x)
    if how.startswith("graph"):
        chain(smcsd, st, lambda: None, lambda x: x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain(smcsd, st, lambda: None, between)
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
    else:
        for _ in range(5):
            got = chain(smcsd, st, lambda: None, between)
        torch.cuda.synchronize()
    for w in ws.values():
        assert smcsd.check_status(w) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_of_one_allocation_are_tensors_of_their_own(smcsd):
    import copy
    import io
    z = torch.randn(6, 500, device="cuda")
    want = {k: host(v).copy() for k, v in smcsd.beam_select(z, 2, 3, 500, 5).items()}
    got = smcsd.beam_select(z, 2, 3, 500, 5)
    for k, t in got.items():
        assert t.data_ptr() % 256 == 0 and t.is_contiguous() and t.shape == (10,) and not t.requires_grad and not t._is_view()
        file = io.BytesIO()
        torch.save(t, file)
        file.seek(0)
        assert np.array_equal(host(torch.load(file)), want[k]) and np.array_equal(host(copy.deepcopy(t)), want[k])
        assert np.array_equal(host(t[1:4]), want[k][1:4]) and np.array_equal(host(t.view(2, 5) + 0), want[k].reshape(2, 5))
    tokens = got["tokens"]
    version = tokens._version
    got["ancestors"].fill_(-7)
    del got, t
    junk = [torch.full((64,), 99, device="cuda", dtype=torch.int32) for _ in range(64)]
    assert np.array_equal(host(tokens), want["tokens"]) and tokens._version == version and len(junk) == 64
    scores = torch.zeros(10, device="cuda", requires_grad=True)
    again = smcsd.beam_select(z, 2, 3, 500, 5)
    (scores * again["scores"]).sum().backward()
    assert np.array_equal(host(scores.grad), want["scores"])
