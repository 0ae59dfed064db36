"""Beam selection, page housekeeping and distillation, as they are measured.

  beam     beam_select                the best continuations of a group's beams over the vocabulary (with one beam: a row's top logits);
           state_reorder, kv_pagetable_remap
                                      the beams' states and page tables follow their ancestors
  pages    kv_free, kv_fork           pages of rejected drafts and finished sequences let go, prompts forked into new sequences
  compact  kv_compact, kv_copy_pages  pages in use moved to the front of the cache
  distill  distill_loss               the draft's loss against a teacher's top logits, and its gradient

``run`` computes each of them in plain torch operations (``own = False``) or by the library (``own = True``). Sizes are those of
the package's workloads: groups of 16 and of 64, vocabularies of 1000, 32000, 32256, 128256 and 151936, 16-token pages, contexts of
2048 and 4096 tokens, hidden states of 2048; head counts, head sizes, the 32768-token context and list lengths are generic.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # four beams of one request over a small vocabulary, with their token histories and tables: latency
        dict(name="beam_1x4", op="beam", G=1, N=4, M=4, V=32000, dtype="bf16", temperature=1.0, done=0, dead=0, states=True, ctx=2048),
        # 8 prompts of 16 beams at a large vocabulary, a quarter of them finished, and their states of 2048
        dict(name="beam_8x16", op="beam", G=8, N=16, M=16, V=128256, dtype="bf16", temperature=1.0, done=4, dead=0, states=True, ctx=2048),
        # float32 logits of an odd vocabulary, the first step after the prompt (one beam alive), twice as many kept as there are beams
        dict(name="beam_f32_16x8", op="beam", G=16, N=8, M=16, V=32257, dtype="f32", temperature=0.75, done=0, dead=7, states=False, ctx=0),
        # the 64 top log-probabilities of a teacher's 2048 rows: what distillation takes
        dict(name="top64_2048", op="beam", G=2048, N=1, M=64, V=128256, dtype="bf16", temperature=1.0, done=0, dead=0, states=False, ctx=0),
        # 16 sequences of 2048 tokens after a verify, two of them replaced
        dict(name="pages_16", op="pages", S=16, N=4, ctx=2048, page=16, tail=5, swap=2),
        # 1024 sequences of up to 32768 tokens in groups of 16, an eighth of them replaced
        dict(name="pages_1024", op="pages", S=1024, N=16, ctx=32768, page=16, tail=64, swap=128),
        # a small cache of one layer with a few pages to move: latency
        dict(name="compact_small", op="compact", S=16, num=600, used=300, moves=40, layers=1, Hkv=2, D=64, page=16, dtype="bf16"),
        # two layers of 16384 pages, 2800 of them to be moved
        dict(name="compact_2_layers", op="compact", S=256, num=16384, used=11000, moves=2800, layers=2, Hkv=8, D=128, page=16, dtype="bf16"),
        # a short float32 batch, the rest of the vocabulary as one event
        dict(name="distill_16x1000", op="distill", R=16, V=1000, K=8, dtype="f32", rest=True, temperature=1.0, idle=1, grad=True),
        # a batch of 4096 tokens at a vocabulary of 32000, some of them padding
        dict(name="distill_4096x32000", op="distill", R=4096, V=32000, K=32, dtype="bf16", rest=True, temperature=2.0, idle=300, grad=True),
        # a batch of 2048 tokens at a large vocabulary: the largest
        dict(name="distill_2048x128256", op="distill", R=2048, V=128256, K=64, dtype="bf16", rest=False, temperature=1.0, idle=0, grad=True),
        # the loss alone, of held-out rows in float32
        dict(name="distill_loss_640", op="distill", R=640, V=151936, K=64, dtype="f32", rest=False, temperature=1.0, idle=0, grad=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def _vocab(rng):
    return rng.choice([1000, 32000, 32256, 128256, 151936, _log_int(rng, 100, 150000), _log_int(rng, 100, 150000)])


def draw(rng):
    op = rng.choice(["beam", "beam", "pages", "compact", "distill", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    b = 4 if dtype == "f32" else 2
    most = 2048 * 128256 * 2 // b  # logits of the largest case
    if op == "beam":
        V = _vocab(rng)
        N = rng.choice([1, 1, 4, 8, 16, 64, _log_int(rng, 2, 64)])
        states = N > 1 and rng.random() < 0.6
        M = N if states else min(V, rng.choice([N, 2 * N, _log_int(rng, 1, 128)]))
        G = max(1, min(_log_int(rng, 1, 2048), (1024 if states else 8192) // N, most // (2 if states else 1) // (N * V)))
        done = rng.choice([0, 0, N // 4])
        return dict(op=op, G=G, N=N, M=M, V=V, dtype=dtype, temperature=rng.choice([1.0, 1.0, 0.75, 1.25]), done=done,
                    dead=rng.choice([0, 0, N - 1 - done]), states=states, ctx=_log_int(rng, 16, 4096) if states else 0)
    if op == "pages":
        S = _log_int(rng, 1, 1024)
        ctx = _log_int(rng, 1, 32768)
        return dict(op=op, S=S, N=min(S, rng.choice([1, 4, 16])), ctx=ctx, page=rng.choice([16, 16, 32, 64]), tail=_log_int(rng, 1, 64),
                    swap=_log_int(rng, 1, S) - 1)
    if op == "compact":
        Hkv, D, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([8, 16, 32])
        layers = rng.choice([1, 1, 2])
        num = min(_log_int(rng, 8, 16384), 16384 * 2 * 8 * 128 * 16 * 2 // (layers * Hkv * D * page * b))
        used = max(1, int(num * rng.uniform(0.1, 0.9)))
        moves = min(int(min(used, num - used) * rng.uniform(0, 0.8)), 2800 * 2 * 8 * 128 * 16 * 2 // (layers * Hkv * D * page * b))
        return dict(op=op, S=_log_int(rng, 1, 256), num=num, used=used, moves=moves, layers=layers, Hkv=Hkv, D=D, page=page, dtype=dtype)
    V = _vocab(rng)
    R = max(1, min(_log_int(rng, 1, 4096), most // V))
    return dict(op=op, R=R, V=V, K=min(V - 1, _log_int(rng, 1, 128)), dtype=dtype, rest=rng.random() < 0.5,
                temperature=rng.choice([1.0, 1.0, 2.0, 0.75]), idle=rng.choice([0, R // 8]), grad=rng.random() < 0.7)


# ------------------------------------------------------------------------------------------------
# sizes that follow from a case
# ------------------------------------------------------------------------------------------------

def _types(case):
    return (torch.float32, 4) if case["dtype"] == "f32" else (torch.bfloat16, 2)


HIDDEN = 2048  # a beam's hidden state


def _spread(n, most, least):
    """n whole numbers of [least, most], the largest first, spread over the upper half of that range: the same ones for every seed."""
    i = np.arange(n, dtype=np.int64)
    return np.maximum(least, most - (i * 2654435761 % 1009) * max(0, most - least) // 2018)


def _page_counts(case):
    """Of a page case: tokens in the cache of each group's prompt and of each sequence, pages of a table row."""
    S, N, page = case["S"], case["N"], case["page"]
    groups = (S + N - 1) // N
    ctx = np.repeat(_spread(groups, case["ctx"], 1), N)[:S]
    return ctx, (case["ctx"] + case["tail"] + page - 1) // page


def work(case):
    op = case["op"]
    if op == "beam":
        _, b = _types(case)
        S = case["G"] * case["N"]
        live = case["G"] * (case["N"] - case["done"] - case["dead"])
        moved = 0
        if case["states"]:
            moved = 2 * S * (case["ctx"] * 4 + HIDDEN * 2 + 4 + _table_pages(case) * 4) + 4 * S * _table_pages(case)
        return {"bytes": live * case["V"] * b + 12 * case["G"] * case["M"] + moved, "flops": 4 * live * case["V"]}
    if op == "pages":
        S = case["S"]
        _, P = _page_counts(case)
        num = _page_number(case)
        return {"bytes": 2 * (8 * S * P + 8 * num) + 16 * S, "flops": 2 * S * P}
    if op == "compact":
        _, b = _types(case)
        page_bytes = case["Hkv"] * case["D"] * case["page"] * b
        entries = case["S"] * _compact_pages(case)
        return {"bytes": 2 * 2 * case["layers"] * case["moves"] * page_bytes + 8 * entries + 8 * case["num"] + 8 * case["moves"], "flops": 0}
    _, b = _types(case)
    read = (case["R"] - case["idle"]) * case["V"] * b
    return {"bytes": read + (case["R"] * case["V"] * b if case["grad"] else 0) + case["R"] * (8 * case["K"] + 8),
            "flops": 8 * case["R"] * case["V"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _randn(shape, dtype, gen, std=1.0):
    out = torch.empty(shape, device=DEV, dtype=dtype)
    flat = out.view(-1)
    step = 1 << 27  # float32 noise of a piece at a time
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at: at + n] = torch.randn(n, device=DEV, generator=gen) * std
    return out


def _table_pages(case):
    return (case["ctx"] + 15) // 16 + 1


def _page_number(case):
    ctx, P = _page_counts(case)
    return case["S"] * P + 64


def _compact_pages(case):
    return max(1, (case["used"] * 5 // 4 + case["S"] - 1) // case["S"])


def _prepare_beam(case, rng, gen):
    dtype, _ = _types(case)
    G, N, V = case["G"], case["N"], case["V"]
    S = G * N
    st = dict(logits=_randn((S, V), dtype, gen, 3.0))
    st["scores"] = -(torch.rand(S, device=DEV, generator=gen) * 4 + 8 * (N > 1))
    order = np.argsort(rng.random((G, N)), axis=1)
    st["finished"] = None
    if case["done"]:
        finished = np.zeros((G, N), np.int32)
        np.put_along_axis(finished, order[:, : case["done"]], 1, 1)
        st["finished"] = _dev(finished.reshape(-1))
    if case["dead"]:
        dead = np.zeros((G, N), bool)
        np.put_along_axis(dead, order[:, N - case["dead"]:], True, 1)
        st["scores"] = torch.where(_dev(dead.reshape(-1)), torch.full_like(st["scores"], NEG), st["scores"])
    st["pad"] = 0
    if case["states"]:
        P = _table_pages(case)
        st["num_pages"] = S * P
        # a group's beams share the first half of their pages
        table = torch.randperm(S * P, device=DEV, generator=gen).to(torch.int32).reshape(S, P)
        head = torch.arange(S, device=DEV) // N * N
        table[:, : P // 2] = table[head, : P // 2]
        st["table"] = table
        st["states"] = [torch.randint(0, V, (S, case["ctx"]), device=DEV, generator=gen, dtype=torch.int32),
                        _randn((S, HIDDEN), torch.bfloat16, gen), torch.rand(S, device=DEV, generator=gen)]
    return st


def _prepare_pages(case, rng, gen):
    S, N, page = case["S"], case["N"], case["page"]
    ctx, P = _page_counts(case)
    num = _page_number(case)
    ids = torch.randperm(num, device=DEV, generator=gen)[: S * P].to(torch.int32).reshape(S, P)
    col = torch.arange(P, device=DEV)
    # what a verify leaves: the pages of the prompt (nine tenths of the context) are the group's, the others a sequence's own
    shared = _dev(ctx * 9 // 10 // page)
    head = torch.arange(S, device=DEV) // N * N
    have = _dev((ctx + case["tail"] + page - 1) // page)
    table = torch.where(col[None] < shared[:, None], ids[head], ids)
    table = torch.where(col[None] < have[:, None], table, torch.full_like(table, -1)).contiguous()
    held = torch.where(table >= 0, table, torch.full_like(table, num)).reshape(-1).long()
    refcount = torch.zeros(num + 1, dtype=torch.int32, device=DEV).index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    keep = ctx + rng.integers(0, case["tail"] + 1, S)
    # the sequences that end are replaced by forks of others, up to the others' prompts
    gone = rng.permutation(S)[: case["swap"]]
    stay = np.setdiff1d(np.arange(S), gone)
    keep[gone] = 0
    parents, lengths = np.arange(S), np.full(S, np.iinfo(np.int32).max)
    if gone.size:
        parents[gone] = rng.choice(stay, gone.size)
        lengths[gone] = ctx[parents[gone]] * 9 // 10
    return dict(table=table, refcount=refcount[:num].contiguous(), keep=_dev(keep.astype(np.int32)),
                parents=_dev(parents.astype(np.int32)), lengths=_dev(lengths.astype(np.int32)), num_pages=num, page=page)


def _prepare_compact(case, rng, gen):
    dtype, _ = _types(case)
    num, used, moves, S = case["num"], case["used"], case["moves"], case["S"]
    P = _compact_pages(case)
    # `moves` pages in use lie behind the first `used`, as many holes before it
    low = rng.permutation(used)[: used - moves]
    high = used + rng.permutation(num - used)[:moves]
    pages = rng.permutation(np.concatenate([low, high]))
    # each page is held once, a fifth of them twice
    held = rng.permutation(np.concatenate([pages, pages[: used // 5]]))[: S * P]
    table = np.full(S * P, -1, np.int64)
    table[: held.size] = held
    table = rng.permutation(table).reshape(S, P)
    refcount = np.bincount(table[table >= 0], minlength=num)
    refcount[pages] = np.maximum(refcount[pages], 1)  # a page that no table holds is held by a prefix cache
    shape = (num, case["Hkv"], case["page"], case["D"])
    caches = [_randn(shape, dtype, gen) for _ in range(2 * case["layers"])]
    return dict(table=_dev(table.astype(np.int32)), refcount=_dev(refcount.astype(np.int32)), caches=caches, num_pages=num)


def _prepare_distill(case, rng, gen):
    dtype, _ = _types(case)
    R, V, K = case["R"], case["V"], case["K"]
    st = dict(logits=_randn((R, V), dtype, gen, 3.0))
    # the teacher agrees with the draft more or less: its list are the top tokens of the draft's logits with noise
    ids = torch.empty(R, K, dtype=torch.int32, device=DEV)
    values = torch.empty(R, K, device=DEV)
    step = max(1, (1 << 26) // V)
    for a in range(0, R, step):
        z = st["logits"][a: a + step].float()
        z = z + torch.randn(z.shape, device=DEV, generator=gen)
        top, at = torch.topk(torch.log_softmax(z, 1), K, dim=1)
        ids[a: a + step], values[a: a + step] = at.int(), top
    st["tokens"], st["values"] = ids, values
    weight = torch.rand(R, device=DEV, generator=gen) + 0.5
    if case["idle"]:
        idle = _dev(rng.permutation(R)[: case["idle"]])
        weight[idle] = 0
        st["tokens"][idle] = -1
    st["weight"] = weight / R
    return st


def prepare(case, seed):
    rng, gen = np.random.default_rng([int(seed), 29]), _gen(seed)
    st = {"beam": _prepare_beam, "pages": _prepare_pages, "compact": _prepare_compact, "distill": _prepare_distill}[case["op"]](case, rng, gen)
    st["case"] = dict(case)
    return st


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------

def _best(x, M):
    """The M largest of each row, ties to the lowest index, in that order: values and indexes."""
    last = torch.topk(x, M, dim=1).values[:, -1:]
    above, tie = x > last, x == last
    room = M - above.sum(1, keepdim=True)
    chosen = above | (tie & (tie.to(torch.int32).cumsum(1, dtype=torch.int32) <= room))
    # M in each row, by rising index; a stable sort keeps that order among equals
    at = chosen.nonzero()[:, 1].reshape(-1, M)
    value, order = torch.sort(x.gather(1, at), dim=1, descending=True, stable=True)
    return value, at.gather(1, order)


def _plain_beam(st):
    case = st["case"]
    G, N, M, V = case["G"], case["N"], case["M"], case["V"]
    score, token, ancestor = [], [], []
    groups = max(1, (1 << 26) // (N * V))  # groups at a time
    for g in range(0, G, groups):
        n = min(groups, G - g)
        rows = slice(g * N, (g + n) * N)
        # 64 bits: beams next to one another in the order
        z = st["logits"][rows].double() / case["temperature"]
        m = z.amax(1, keepdim=True)
        lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
        base = st["scores"][rows].double()[:, None]
        x = z - lse + base
        if st["finished"] is not None:
            over = st["finished"][rows, None] != 0
            only = torch.full_like(x, NEG)
            only[:, 0] = base[:, 0]  # the one candidate of a finished beam
            x = torch.where(over, only, x)
        value, at = _best(x.reshape(n, N * V), M)
        beam, v = at // V, at % V
        none = value == NEG
        ended = torch.zeros_like(none)
        if st["finished"] is not None:
            ended = (st["finished"][rows].reshape(n, N).gather(1, beam) != 0) & ~none
            v = torch.where(ended, torch.full_like(v, st["pad"]), v)
        v = torch.where(none, torch.full_like(v, st["pad"]), v)
        beam = torch.where(none, torch.zeros_like(beam), beam)
        score.append(value.float().reshape(-1))
        token.append(v.int().reshape(-1))
        ancestor.append(beam.int().reshape(-1))
    out = dict(tokens=torch.cat(token), ancestors=torch.cat(ancestor), scores=torch.cat(score))
    if case["states"]:
        parent = torch.arange(G * N, device=DEV) // N * N + out["ancestors"].long()
        out["states"] = [s[parent] for s in st["states"]]
        table = out["table"] = st["table"][parent]
        out["refcount"] = torch.zeros(st["num_pages"], dtype=torch.int32, device=DEV).index_add_(
            0, table.reshape(-1), torch.ones(table.numel(), dtype=torch.int32, device=DEV))
    return out


def _plain_counts(table, num, sign, out):
    """out (with a place for -1 at its end) with sign added for every entry of the table."""
    held = torch.where(table >= 0, table, torch.full_like(table, num)).reshape(-1)
    return out.index_add_(0, held, torch.full_like(held, sign))


def _plain_pages(st):
    table, page, num = st["table"], st["page"], st["num_pages"]
    col = torch.arange(table.shape[1], device=DEV)[None]
    pages = lambda n: ((n.long() + page - 1) // page)[:, None]  # noqa: E731
    none = torch.full_like(table, -1)
    freed = torch.where(col < pages(st["keep"]), table, none)
    forked = torch.where(col < pages(st["lengths"]), freed[st["parents"].long()], none)
    count = torch.cat([st["refcount"], st["refcount"].new_zeros(1)])
    count = _plain_counts(freed, num, 1, _plain_counts(table, num, -1, count))
    freed_count = count[:num].clone()
    count = _plain_counts(forked, num, 1, _plain_counts(freed, num, -1, count))
    return dict(freed=freed, freed_refcount=freed_count, forked=forked, forked_refcount=count[:num])


def _plain_compact(st):
    case, num = st["case"], st["num_pages"]
    table, ref = st["table"], st["refcount"]
    held = ref > 0
    used = held.sum()
    at = torch.arange(num, device=DEV)
    hole, mover = ~held & (at < used), held & (at >= used)
    # the i-th hole takes the i-th page from behind; there is room for half of the pages in each list
    half = num // 2
    order = lambda which: torch.where(which, which.long().cumsum(0) - 1, torch.full_like(at, half))  # noqa: E731
    lists = torch.full((2, half + 1), -1, dtype=torch.int64, device=DEV)
    src, dst = lists[0].index_copy(0, order(mover), at)[:half], lists[1].index_copy(0, order(hole), at)[:half]
    n = case["moves"]
    to = torch.cat([at, at.new_full((1,), -1)]).index_copy(0, src[:n], dst[:n])
    table_out = to[torch.where(table >= 0, table.long(), torch.full_like(table, num).long())].int()
    ref_out = ref.index_copy(0, dst[:n], ref[src[:n]]).index_fill(0, src[:n], 0)
    for cache in st["caches"]:
        cache[dst[:n]] = cache[src[:n]]
    return dict(table=table_out, refcount=ref_out, src=src.int(), dst=dst.int(),
                counts=torch.stack([mover.sum(), used]).int(), caches=st["caches"])


def _plain_distill(st):
    case = st["case"]
    R, V, T = case["R"], case["V"], case["temperature"]
    loss, grads = [], []
    step = max(1, (1 << 28) // V)
    for a in range(0, R, step):
        rows = slice(a, min(R, a + step))
        z = st["logits"][rows].float() / T
        there = st["tokens"][rows] >= 0
        ids = st["tokens"][rows].long().clamp(min=0)
        some = there.any(1)
        value = torch.where(there, st["values"][rows], torch.full_like(st["values"][rows], NEG))
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        lse = m + torch.log(total)
        logq = z.gather(1, ids) - lse
        if case["rest"]:
            logp = value
            p = torch.exp(logp)
            rest = (1 - p.double().sum(1)).clamp(min=0).float()
        else:
            top = torch.where(some, value.amax(1), torch.zeros_like(m[:, 0]))[:, None]
            logp = value - top - torch.log(torch.exp(value - top).sum(1, keepdim=True))
            p = torch.exp(logp)
        each = torch.where(p > 0, p * (logp - logq), torch.zeros_like(p)).sum(1)
        if case["rest"]:
            away = e.scatter(1, torch.where(there, ids, ids[:, :1]), 0.0)  # a list's first entry is there, or none is
            rest_q = torch.where(some, away.sum(1) / total[:, 0], torch.ones_like(rest))
            each = each + torch.where(rest > 0, rest * (torch.log(rest) - torch.log(rest_q)), torch.zeros_like(rest))
        loss.append(torch.where(some, each, torch.zeros_like(each)))
        if case["grad"]:
            w = torch.where(some, st["weight"][rows], torch.zeros_like(each))[:, None] / T
            q = e / total
            p = torch.where(there, p, torch.zeros_like(p))
            if case["rest"]:
                mass = p.sum(1, keepdim=True) + rest[:, None]
                grad = q * (mass - (rest / rest_q)[:, None])
                grad.scatter_(1, torch.where(there, ids, ids[:, :1]), torch.where(there, q.gather(1, ids) * mass - p,
                                                                                  (q.gather(1, ids) * mass - p)[:, :1]))
            else:
                grad = q.scatter_add(1, ids, -p)
            grads.append((grad * w).to(st["logits"].dtype))
    return dict(loss=torch.cat(loss), grad=torch.cat(grads) if case["grad"] else None)


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------

_kept = {}  # one workspace for each operation and size, as a program keeps them


def _workspace(lib, op, *sizes):
    key = (op, *sizes)
    if key not in _kept:
        _kept[key] = lib.Workspace(op, *sizes)
    return _kept[key]


def _own_run(st):
    import smc_reweight_resample_gb300 as lib

    case, op = st["case"], st["case"]["op"]
    if op == "beam":
        G, N, M, V = case["G"], case["N"], case["M"], case["V"]
        out = lib.beam_select(st["logits"], G, N, V, M, temperature=case["temperature"], scores=st["scores"], finished=st["finished"],
                              pad_token=st["pad"], ws=_workspace(lib, lib.OP_BEAM_SELECT, G * N, N, V))
        got = dict(tokens=out["tokens"], ancestors=out["ancestors"], scores=out["scores"])
        if case["states"]:
            got["states"] = lib.state_reorder(st["states"], out["ancestors"], G, N, ws=_workspace(lib, lib.OP_STATE_REORDER, 1))
            got["table"], got["refcount"] = lib.kv_pagetable_remap(out["ancestors"], None, G, N, st["table"], st["table"].shape[1],
                                                                   st["num_pages"], ws=_workspace(lib, lib.OP_PAGETABLE_REMAP, G))
        return got
    if op == "pages":
        ws = _workspace(lib, lib.OP_KV_FORK, 1)
        freed, count = lib.kv_free(st["table"], st["refcount"], st["keep"], st["page"], ws=ws)
        forked, forked_count = lib.kv_fork(freed, count, st["parents"], st["page"], lengths=st["lengths"], ws=ws)
        return dict(freed=freed, freed_refcount=count, forked=forked, forked_refcount=forked_count)
    if op == "compact":
        ws = _workspace(lib, lib.OP_KV_COMPACT, case["S"], 0, st["num_pages"])
        got = lib.kv_compact(st["table"], st["refcount"], ws=ws)
        lib.kv_copy_pages(st["caches"], got["src"], got["dst"], count=got["counts"], ws=ws)
        return dict(table=got["table_out"], refcount=got["refcount_out"], src=got["src"], dst=got["dst"], counts=got["counts"],
                    caches=st["caches"])
    loss, grad = lib.distill_loss(st["logits"], st["tokens"], st["values"], case["V"], temperature=case["temperature"], rest=case["rest"],
                                  weight=st["weight"], grad=case["grad"], ws=_workspace(lib, lib.OP_DISTILL_LOSS, 1))
    return dict(loss=loss, grad=grad)


def run(state):
    if own:
        return _own_run(state)
    return {"beam": _plain_beam, "pages": _plain_pages, "compact": _plain_compact, "distill": _plain_distill}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# 64 bits, from the definitions
# ------------------------------------------------------------------------------------------------

def _exact_beam(st):
    """The scores, group by group: of every beam its M best tokens, of those the M best."""
    case = st["case"]
    G, N, M, V = case["G"], case["N"], case["M"], case["V"]
    scores = torch.full((G, M), NEG, dtype=torch.float64, device=DEV)
    for g in range(G):
        rows = st["logits"][g * N: (g + 1) * N].double()
        logp = torch.log_softmax(rows / case["temperature"], 1) + st["scores"][g * N: (g + 1) * N, None].double()
        best = [logp[i].sort(descending=True).values[:M] if st["finished"] is None or not bool(st["finished"][g * N + i])
                else st["scores"][g * N + i: g * N + i + 1].double() for i in range(N)]
        best = torch.cat(best).sort(descending=True).values[:M]
        scores[g, : best.numel()] = best
    out = dict(tokens=None, ancestors=None, scores=scores.reshape(-1))
    if case["states"]:
        out.update(states=[None] * len(st["states"]), table=None, refcount=None)
    return out


def _exact_compact(st):
    ref = st["refcount"].cpu().numpy()
    used = int((ref > 0).sum())
    dst = [i for i in range(used) if ref[i] == 0]
    src = [i for i in range(used, ref.size) if ref[i] > 0]
    caches = []
    for cache in st["caches"]:
        c = cache.double()
        for a, b in zip(src, dst):
            c[b] = c[a].clone()
        caches.append(c)
    return dict(table=None, refcount=None, src=None, dst=None, counts=None, caches=caches)


def _exact_distill(st):
    case = st["case"]
    R, V, T = case["R"], case["V"], case["temperature"]
    loss = torch.zeros(R, dtype=torch.float64, device=DEV)
    grad = torch.zeros(R, V, dtype=torch.float64, device=DEV) if case["grad"] else None
    step = max(1, (1 << 25) // V)
    for a in range(0, R, step):
        b = min(R, a + step)
        tokens = st["tokens"][a:b].long()
        some = tokens[:, 0] >= 0
        ids = torch.where(tokens >= 0, tokens, torch.zeros_like(tokens))
        logq = torch.log_softmax(st["logits"][a:b].double() / T, 1)
        value = st["values"][a:b].double()
        target = torch.zeros(b - a, V, dtype=torch.float64, device=DEV)
        lists = torch.zeros(b - a, V, dtype=torch.bool, device=DEV).scatter_(1, ids, True)
        q = logq.exp()
        p = value.exp() if case["rest"] else torch.softmax(value, 1)
        target.scatter_add_(1, ids, p)
        part = (p * (p.log() - logq.gather(1, ids))).sum(1)
        d = q * target.sum(1, keepdim=True) - target
        if case["rest"]:
            over = (1 - p.sum(1)).clamp(min=0)
            out = q.masked_fill(lists, 0.0).sum(1)
            part = part + torch.special.xlogy(over, over / out)
            d = d + over[:, None] * (q - (q / out[:, None]).masked_fill(lists, 0.0))
        loss[a:b] = torch.where(some, part, torch.zeros_like(part))
        if grad is not None:
            grad[a:b] = d * torch.where(some, st["weight"][a:b].double(), torch.zeros_like(part))[:, None] / T
    return dict(loss=loss, grad=grad)


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers
    st = prepare(case, seed)
    return {"beam": _exact_beam, "compact": _exact_compact, "distill": _exact_distill}[case["op"]](st)
