"""The cached-attention and logits operators of one speculative step, as they are measured.

A step of speculative decoding with a paged KV cache runs, around the verify that the library already has:

  slots    kv_slot_map    page tables, copy-on-write pages and slot numbers of the step's new tokens, from request lengths
  append   kv_append      the new tokens' keys and values into their slots (and the shared partial pages' copies)
  attn     tree_mask, tree_attention
                          the drafted tokens (a chain or a tree for each sequence) over the cache and over their ancestors
  logits   logits_process repetition / presence / frequency penalties, biases and grammar masks before sampling or verify

``run`` computes each of them in plain torch operations in 32 bits (``own = False``) or by the library (``own = True``).
Sizes are those of the package's workloads: 8 x 16 particles with K=4 and a 2048-token context, 4 x 64 particles with
K=8 and a 4096-token context, 16-token pages, 16 sequences with K=4, 64 ragged sequences of up to 20 drafts, vocabularies
of 1000, 32000, 32256, 128256 and 151936; head counts, head sizes and the 32768-token context are generic.
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
        # one new token for each of 16 requests: what a plain decode step asks of the page tables
        dict(name="slots_16x1", op="slots", G=16, N=1, T=1, ctx=2048, page=16, ragged=False),
        # 4 x 64 particles after a resampling (shared pages, copies on write), K=8 drafts and the last token
        dict(name="slots_256x9", op="slots", G=4, N=64, T=9, ctx=4096, page=16, ragged=False),
        # the keys and values of 8 x 16 particles' K+1 tokens, with the copies of their shared last pages
        dict(name="append_128x5", op="append", G=8, N=16, T=5, ctx=2048, page=16, ragged=False, Hkv=8, D=128, dtype="bf16"),
        # 16 prompts of up to 2048 tokens written at once
        dict(name="append_prompts", op="append", G=16, N=1, T=2048, ctx=0, page=16, ragged=True, Hkv=8, D=128, dtype="bf16"),
        # a single token of a single request: latency
        dict(name="attn_1x1", op="attn", G=1, N=1, T=1, ctx=517, page=16, ragged=False, tree=False, shared=0.0, Hq=32, Hkv=8, D=128,
             dtype="bf16"),
        # 16 requests of ragged lengths, chains of K+1=5, heads of 64 that share no keys
        dict(name="attn_16x5_d64", op="attn", G=16, N=1, T=5, ctx=2048, page=16, ragged=False, tree=False, shared=0.0, Hq=16, Hkv=16, D=64,
             dtype="bf16"),
        # 8 x 16 particles with K=4: a group's particles share the pages of their prompt and of common ancestors
        dict(name="attn_smc_8x16", op="attn", G=8, N=16, T=5, ctx=2048, page=16, ragged=False, tree=False, shared=0.9, Hq=32, Hkv=8, D=128,
             dtype="bf16"),
        # trees of up to 64 drafted tokens over long contexts: the largest
        dict(name="attn_tree_8x64", op="attn", G=8, N=1, T=64, ctx=32768, page=16, ragged=True, tree=True, shared=0.0, Hq=64, Hkv=8, D=128,
             dtype="bf16"),
        # 64 requests with ragged chains of up to 21 tokens, no page shared
        dict(name="attn_64x21", op="attn", G=64, N=1, T=21, ctx=4096, page=16, ragged=True, tree=False, shared=0.0, Hq=32, Hkv=8, D=128,
             dtype="bf16"),
        # the float32 form at a small size
        dict(name="attn_f32", op="attn", G=4, N=1, T=3, ctx=1000, page=16, ragged=False, tree=True, shared=0.0, Hq=8, Hkv=4, D=64, dtype="f32"),
        # a float32 step of 4 sequences at a vocabulary of 1000: the smallest logits
        dict(name="logits_4x3", op="logits", G=4, N=1, T=3, V=1000, hist=200, nbias=5, grammar=True, ragged=False, tree=False, dtype="f32"),
        # the logits of 8 x 16 particles' K+1 positions, penalties, biases and a grammar
        dict(name="logits_128x5", op="logits", G=128, N=1, T=5, V=128256, hist=2048, nbias=32, grammar=True, ragged=False, tree=False,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["slots", "append", "attn", "attn", "attn", "logits"])
    if op == "slots":
        G, N = _log_int(rng, 1, 16), rng.choice([1, 4, 16, 64, 7])
        return dict(op=op, G=G, N=N, T=_log_int(rng, 1, 64), ctx=_log_int(rng, 1, 4096), page=rng.choice([8, 16, 32, 64]),
                    ragged=rng.random() < 0.5)
    if op == "append":
        T = _log_int(rng, 1, 2048)
        N = rng.choice([1, 1, 4, 16]) if T <= 64 else 1
        G = max(1, min(_log_int(rng, 1, 128 // N), 32768 // T))
        return dict(op=op, G=G, N=N, T=T, ctx=_log_int(rng, 1, 2048) - 1, page=rng.choice([8, 16, 32, 64]), ragged=rng.random() < 0.5,
                    Hkv=rng.choice([1, 2, 4, 8, 5]), D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "attn":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 4, 5, 8])
        T = _log_int(rng, 1, 64 if dtype == "bf16" else 8)
        N = rng.choice([1, 1, 4, 16])
        ctx = _log_int(rng, 1, 32768 if dtype == "bf16" else 2048)
        # rows x keys of the call, as a share of the largest listed case's
        most = 8 * 64 * 64 * 32768 if dtype == "bf16" else 1 << 24
        keys = 1 << (18 if dtype == "bf16" else 16)
        if N * ctx > keys or N * T * Hq * ctx > most:
            N = 1
        G = max(1, min(_log_int(rng, 1, 64), most // (N * T * Hq * ctx), keys // (N * ctx)))
        return dict(op=op, G=G, N=N, T=T, ctx=ctx, page=rng.choice([8, 16, 32, 64]), ragged=rng.random() < 0.5, tree=rng.random() < 0.5,
                    shared=rng.choice([0.0, 0.5, 0.9]) if N > 1 else 0.0, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype)
    V = rng.choice([1000, 32000, 32256, 128256, 151936, _log_int(rng, 100, 150000)])
    T = _log_int(rng, 1, 21)
    G = max(1, min(_log_int(rng, 1, 128), 640 * 128256 // (2 * T * V)))
    return dict(op=op, G=G, N=1, T=T, V=V, hist=_log_int(rng, 1, 4096), nbias=_log_int(rng, 1, 64), grammar=rng.random() < 0.6,
                ragged=rng.random() < 0.5, tree=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------------------------------------
# sizes that follow from a case
# ------------------------------------------------------------------------------------------------

def _spread(n, most, least):
    """n whole numbers of [least, most], the largest first, spread over the upper half of that range: the same ones for every seed."""
    i = np.arange(n, dtype=np.int64)
    return np.maximum(least, most - (i * 2654435761 % 1009) * max(0, most - least) // 2018)


def _counts(case):
    """New tokens (nodes) of each sequence."""
    S = case["G"] * case["N"]
    return _spread(S, case["T"], 1) if case["ragged"] else np.full(S, case["T"], np.int64)


def _contexts(case):
    """Tokens in the cache, for each group (a group's particles have equally many)."""
    return _spread(case["G"], case["ctx"], min(1, case["ctx"]))


def _types(case):
    return (torch.float32, 4) if case["dtype"] == "f32" else (torch.bfloat16, 2)


def work(case):
    S, page = case["G"] * case["N"], case.get("page", 16)
    n = _counts(case)
    R = int(n.sum())
    if case["op"] == "slots":
        P = (case["ctx"] + case["T"] + page - 1) // page
        pages = S * (P + 1)
        return {"bytes": 8 * S * P + 8 * pages + 8 * R + 16 * S, "flops": S * P + pages + R}
    if case["op"] == "append":
        _, b = _types(case)
        part = int((np.repeat(_contexts(case), case["N"]) % page).sum()) if case["N"] > 1 else 0
        return {"bytes": (R + part) * case["Hkv"] * case["D"] * b * 4 + 8 * R, "flops": 0}
    if case["op"] == "attn":
        _, b = _types(case)
        c = _contexts(case)
        alike = (case["shared"] * c / page).astype(np.int64) * page
        keys = int((c - alike).sum()) * case["N"] + int(alike.sum()) + R
        c = np.repeat(c, case["N"])
        seen = int((n * c).sum()) + int((n * (n + 1) // 2).sum())
        return {"bytes": keys * case["Hkv"] * case["D"] * 2 * b + 2 * R * case["Hq"] * case["D"] * b + 4 * R * case["Hq"],
                "flops": 4 * seen * case["Hq"] * case["D"]}
    _, b = _types(case)
    V = case["V"]
    return {"bytes": 2 * R * V * b + (R * ((V + 31) // 32) * 4 if case["grammar"] else 0) + 4 * int(_spread(S, case["hist"], 0).sum()),
            "flops": R * V}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _randn(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * std).to(dtype)


def _parents(counts, rng):
    """For each node of each sequence the node that it follows, -1 for a first one: mostly shallow trees."""
    at = np.concatenate([np.arange(c) for c in counts])
    back = np.minimum(1 + (rng.random(at.size) ** 3 * 16).astype(np.int64), at + 1)
    return (at - back).astype(np.int32)


def _tables(case, rng, gen):
    """Page tables as a step finds them: a group's sequences share their leading pages, ids are scattered."""
    G, N, T, page = case["G"], case["N"], case["T"], case["page"]
    S, P = G * N, (case["ctx"] + T + page - 1) // page
    num = S * (P + 1)
    own_pages = torch.randperm(num, device=DEV, generator=gen)[: S * P].to(torch.int32).reshape(S, P)
    return own_pages, S, P, num, rng.permutation(_contexts(case))


def prepare(case, seed):
    rng, gen = np.random.default_rng([int(seed), 17]), _gen(seed)
    op, page = case["op"], case.get("page", 16)
    counts = _counts(case)
    S, T = case["G"] * case["N"], case["T"]
    st = dict(case=dict(case), S=S, T=T, N=case["N"], R=int(counts.sum()), page=page)
    st["offsets"] = _dev(_offsets(counts)) if case["ragged"] else None
    if op == "logits":
        dtype, _ = _types(case)
        V, R = case["V"], st["R"]
        st.update(V=V, logits=_randn((R, V), dtype, gen, 3.0))
        # a text repeats itself: low token ids come often
        hist = rng.permutation(_spread(S, case["hist"], 0))
        st["hist_offsets"] = _dev(_offsets(hist))
        st["hist_tokens"] = _dev((rng.random(int(hist.sum())) ** 4 * V).astype(np.int32))
        st["node_tokens"] = _dev((rng.random(R) ** 4 * V).astype(np.int32))
        st["parents"] = _dev(_parents(counts, rng)) if case["tree"] else None
        st["repetition"] = _dev(rng.uniform(1.0, 1.3, S).astype(np.float32))
        st["presence"] = _dev(rng.uniform(0.0, 0.6, S).astype(np.float32))
        st["frequency"] = _dev(rng.uniform(0.0, 0.3, S).astype(np.float32))
        nb = min(case["nbias"], V)
        st["bias_offsets"] = _dev(np.arange(S + 1, dtype=np.int32) * nb)
        # distinct tokens for each sequence
        first = rng.integers(0, V, (S, 1))
        st["bias_tokens"] = _dev(((first + np.arange(nb) * max(1, V // nb)) % V).astype(np.int32).reshape(-1))
        st["bias_values"] = _dev(rng.normal(0, 2, S * nb).astype(np.float32))
        st["allowed"] = None
        if case["grammar"]:
            # a third of the rows is free, the others allow a few tokens in a hundred (and always some)
            W = (V + 31) // 32
            word = lambda: torch.randint(-(1 << 31), 1 << 31, (R, W), device=DEV, generator=gen, dtype=torch.int64)  # noqa: E731
            few = word() & word() & word() & word() & word()
            few[:, 0] |= 2
            free = torch.rand((R, 1), device=DEV, generator=gen) < 0.33
            st["allowed"] = torch.where(free, torch.full_like(few, -1), few).to(torch.int32)
        return st

    table, S, P, num, ctx = _tables(case, rng, gen)
    st.update(P=P, num_pages=num)
    ctx_s = np.repeat(ctx, case["N"])
    st["ctx_len"] = _dev(ctx_s.astype(np.int32))
    col = torch.arange(P, device=DEV)
    if op == "attn":
        dtype, _ = _types(case)
        alike = _dev((case["shared"] * ctx_s / page).astype(np.int64))
        head = torch.arange(S, device=DEV) // case["N"] * case["N"]
        table = torch.where(col[None] < alike[:, None], table[head], table)
        have = _dev((ctx_s + counts + page - 1) // page)
        st["table"] = torch.where(col[None] < have[:, None], table, torch.full_like(table, -1)).contiguous()
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        st["q"] = _randn((st["R"], Hq, D), dtype, gen, 2.0)
        st["k_cache"] = _randn((num, Hkv, page, D), dtype, gen)
        st["v_cache"] = _randn((num, Hkv, page, D), dtype, gen)
        st["parents"] = _dev(_parents(counts, rng)) if case["tree"] else None
        st["scale"] = 1.0 / math.sqrt(D)
        return st

    # a group after a resampling: each sequence holds its ancestor's pages, the partly filled last one too
    a = _dev(rng.integers(0, case["N"], S)) + torch.arange(S, device=DEV) // case["N"] * case["N"]
    have = _dev((ctx_s + page - 1) // page)
    table = torch.where(col[None] < have[:, None], table[a], torch.full_like(table, -1)).contiguous()
    held = torch.where(table >= 0, table, torch.full_like(table, num)).reshape(-1).long()
    refcount = torch.zeros(num + 1, dtype=torch.int32, device=DEV)
    refcount.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    st.update(table=table, refcount=refcount[:num].contiguous())
    if op == "append":
        # the slots and page copies that kv_slot_map gives for this step
        m = _plain_slots(st)
        st.update(slots=m["slots"], copy_src=m["copy_src"], copy_dst=m["copy_dst"])
        dtype, _ = _types(case)
        Hkv, D = case["Hkv"], case["D"]
        # keys and values as slices of one projection's output, token by token
        st["kv"] = _randn((st["R"], 2, Hkv, D), dtype, gen)
        st["k_cache"] = _randn((num, Hkv, page, D), dtype, gen)
        st["v_cache"] = _randn((num, Hkv, page, D), dtype, gen)
    return st


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------

def _row_maps(st):
    """For each row its sequence and its number within the sequence; and the rows of each sequence, padded to T."""
    S, T, R = st["S"], st["T"], st["R"]
    if st["offsets"] is None:
        row = torch.arange(R, device=DEV)
        return row // T, row % T, row.reshape(S, T)
    off = st["offsets"].long()
    seq = torch.repeat_interleave(torch.arange(S, device=DEV), off[1:] - off[:-1], output_size=R)
    return seq, torch.arange(R, device=DEV) - off[seq], (off[:-1, None] + torch.arange(T, device=DEV)).clamp(max=R - 1)


def _new_counts(st):
    S, T = st["S"], st["T"]
    if st["offsets"] is None:
        return torch.full((S,), T, device=DEV, dtype=torch.int64)
    return (st["offsets"][1:] - st["offsets"][:-1]).long()


def _plain_slots(st):
    S, P, page, num = st["S"], st["P"], st["page"], st["num_pages"]
    table, ref = st["table"].long(), st["refcount"].long()
    c, n = st["ctx_len"].long(), _new_counts(st)
    col = torch.arange(P, device=DEV)[None]
    first, end = (c // page)[:, None], ((c + n + page - 1) // page)[:, None]
    written = (col >= first) & (col < end) & (n > 0)[:, None]
    shared = (table >= 0) & (ref[table.clamp(min=0)] > 1) & written
    need = written & (table < 0) | shared
    rank = (need.reshape(-1).long().cumsum(0) - 1).reshape(S, P)
    free = ref == 0
    at = torch.where(free, free.long().cumsum(0) - 1, torch.full_like(ref, num))
    pages = torch.empty(num + 1, dtype=torch.int64, device=DEV).index_copy_(0, at, torch.arange(num, device=DEV))
    new = pages[rank.clamp(min=0)]
    out = torch.where(need, new, table)
    up = torch.where(need, new, torch.full_like(new, num)).reshape(-1)
    down = torch.where(shared, table, torch.full_like(table, num)).reshape(-1)
    one = torch.ones_like(up)
    ref_out = torch.cat([ref, ref.new_zeros(1)]).index_add_(0, up, one).index_add_(0, down, -one)[:num]
    seq, i, _ = _row_maps(st)
    pos = c[seq] + i
    slots = out[seq, pos // page] * page + pos % page
    at = first.clamp(max=P - 1)
    copied = (shared.gather(1, at) & (c % page > 0)[:, None])[:, 0]
    none = torch.full((S,), -1, device=DEV, dtype=torch.int64)
    return dict(table_out=out.int(), refcount_out=ref_out.int(), slots=slots,
                copy_src=torch.where(copied, table.gather(1, at)[:, 0], none).int(),
                copy_dst=torch.where(copied, out.gather(1, at)[:, 0], none).int())


def _plain_append(st):
    page = st["page"]
    src, dst = st["copy_src"].long(), st["copy_dst"].long()
    part = (torch.arange(page, device=DEV)[None] < (st["ctx_len"].long() % page)[:, None]) & (src >= 0)[:, None]
    slot = st["slots"]
    # the page that each sequence's first new token goes to, no other's: where nothing is copied it is written with itself
    first = torch.arange(st["S"], device=DEV) * st["T"] if st["offsets"] is None else st["offsets"][:-1].long()
    to = torch.where(dst >= 0, dst, slot[first] // page)
    for cache, new in ((st["k_cache"], st["kv"][:, 0]), (st["v_cache"], st["kv"][:, 1])):
        if st["N"] > 1:
            cache[to] = torch.where(part[:, None, :, None], cache[src.clamp(min=0)], cache[to])
        cache[slot // page, :, slot % page] = new
    return dict(k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_seen(st, rows):
    """[S, T, T]: whether node t sees node j (itself and those that it follows)."""
    S, T = st["S"], st["T"]
    n = _new_counts(st)
    j = torch.arange(T, device=DEV)
    if st["parents"] is None:
        seen = (j[None] <= j[:, None])[None].expand(S, T, T)
    else:
        parent = torch.where(j[None] < n[:, None], st["parents"][rows].long(), torch.full_like(rows, -1))
        step = (parent[:, :, None] == j).float() + torch.eye(T, device=DEV)
        # a node's path is unique, so any positive entry of the T-th power is an ancestor
        seen = torch.linalg.matrix_power(step, T) > 0
    return seen & (j[None, None] < n[:, None, None])


def _plain_attn(st):
    case, S, T, N = st["case"], st["S"], st["T"], st["N"]
    Hq, Hkv, D, P, page = case["Hq"], case["Hkv"], case["D"], st["P"], st["page"]
    g, L = Hq // Hkv, P * page
    seq, t, rows = _row_maps(st)
    c, n = st["ctx_len"].long(), _new_counts(st)
    ids = st["table"].long().clamp(min=0)
    pos = torch.arange(L, device=DEV)
    there = pos[None] < (c + n)[:, None]
    K = st["k_cache"][ids].permute(0, 2, 1, 3, 4).reshape(S, Hkv, L, D).float()
    V = st["v_cache"][ids].permute(0, 2, 1, 3, 4).reshape(S, Hkv, L, D).float()
    V = torch.where(there[:, None, :, None], V, V.new_zeros(()))
    q = st["q"][rows].float().reshape(S, T, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, g * T, D)
    z = (q @ K.transpose(2, 3)).reshape(S, Hkv, g, T, L) * st["scale"]
    node = pos[None] - c[:, None]
    tree = _plain_seen(st, rows)
    sees = (node < 0)[:, None] | (tree.gather(2, node.clamp(0, T - 1)[:, None].expand(S, T, L)) & there[:, None] & (node >= 0)[:, None])
    z = torch.where(sees[:, None, None], z, z.new_full((), NEG))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == NEG, torch.zeros_like(m), m))
    total = e.sum(-1, keepdim=True)
    o = (e.reshape(S, Hkv, g * T, L) @ V).reshape(S, Hkv, g, T, D) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (m + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(S, T, Hq, D)[seq, t]
    return dict(out=o.to(st["q"].dtype), lse=lse.permute(0, 3, 1, 2).reshape(S, T, Hq)[seq, t])


def _plain_logits(st):
    S, T, V, R = st["S"], st["T"], st["V"], st["R"]
    seq, t, rows = _row_maps(st)
    ho = st["hist_offsets"].long()
    nh = st["hist_tokens"].numel()
    hseq = torch.repeat_interleave(torch.arange(S, device=DEV), ho[1:] - ho[:-1], output_size=nh)
    count = torch.zeros(S * V, device=DEV).index_add_(0, hseq * V + st["hist_tokens"].long(), torch.ones(nh, device=DEV)).reshape(S, V)[seq]
    # the drafted tokens on a row's own path, itself among them
    seen = _plain_seen(st, rows)[seq, t]
    token = st["node_tokens"].long()[rows][seq]
    count.scatter_add_(1, token, seen.float())
    z = st["logits"].float()
    hit = count > 0
    rep = st["repetition"][seq][:, None]
    z = torch.where(hit, torch.where(z > 0, z / rep, z * rep), z)
    z = z - st["frequency"][seq][:, None] * count - st["presence"][seq][:, None] * hit
    nb = st["bias_tokens"].numel() // S
    z.scatter_add_(1, st["bias_tokens"].long().reshape(S, nb)[seq], st["bias_values"].reshape(S, nb)[seq])
    if st["allowed"] is not None:
        bit = (st["allowed"][:, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
        z = torch.where(bit.reshape(R, -1)[:, :V] != 0, z, z.new_full((), NEG))
    return dict(out=z.to(st["logits"].dtype))


# ------------------------------------------------------------------------------------------------
# the library's calls
# ------------------------------------------------------------------------------------------------

_kept = {}  # one workspace for each operation and size, as a program keeps them


def _workspace(lib, key, make):
    if key not in _kept:
        _kept[key] = make()
    return _kept[key]


def _own_run(st):
    import smc_reweight_resample_gb300 as lib

    case, S, T, op = st["case"], st["S"], st["T"], st["case"]["op"]
    if op == "slots":
        ws = _workspace(lib, (op, S, st["num_pages"]), lambda: lib.Workspace(lib.OP_KV_SLOT_MAP, S, 0, st["num_pages"]))
        return lib.kv_slot_map(st["ctx_len"], st["table"], st["refcount"], S, T, st["page"], new_offsets=st["offsets"], rows=st["R"], ws=ws)
    if op == "append":
        ws = _workspace(lib, op, lambda: lib.Workspace(lib.OP_KV_APPEND, 1))
        k, v = lib.kv_append(st["kv"][:, 0], st["kv"][:, 1], st["slots"], st["k_cache"], st["v_cache"], ctx_len=st["ctx_len"],
                             copy_src=st["copy_src"], copy_dst=st["copy_dst"], ws=ws)
        return dict(k_cache=k, v_cache=v)
    mask = None
    if st["parents"] is not None:
        ws = _workspace(lib, "mask", lambda: lib.Workspace(lib.OP_TREE_MASK, 1))
        mask = lib.tree_mask(st["parents"], S, T, node_offsets=st["offsets"], ws=ws)
    if op == "attn":
        ws = _workspace(lib, (op, S, st["N"], T, case["Hq"], case["Hkv"], case["D"]),
                        lambda: lib.TreeAttentionWorkspace(S, st["N"], T, case["Hq"], case["Hkv"], case["D"]))
        out, lse = lib.tree_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx_len"], S, T, st["scale"], N=st["N"],
                                      node_offsets=st["offsets"], mask=mask, ws=ws)
        return dict(out=out, lse=lse)
    ws = _workspace(lib, op, lambda: lib.Workspace(lib.OP_LOGITS_PROCESS, 1))
    out = lib.logits_process(st["logits"], S, T, st["V"], node_offsets=st["offsets"], node_tokens=st["node_tokens"], mask=mask,
                             hist_tokens=st["hist_tokens"], hist_offsets=st["hist_offsets"], repetition=st["repetition"],
                             presence=st["presence"], frequency=st["frequency"], bias_tokens=st["bias_tokens"],
                             bias_values=st["bias_values"], bias_offsets=st["bias_offsets"], allowed=st["allowed"], ws=ws)
    return dict(out=out)


def run(state):
    if own:
        return _own_run(state)
    return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attn, "logits": _plain_logits}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# 64 bits, from the definitions, one sequence at a time
# ------------------------------------------------------------------------------------------------

def _paths(parents, n, chain):
    """For each of n nodes the list of the nodes that it sees."""
    got = []
    for t in range(n):
        path, at = [], t
        while at >= 0:
            path.append(at)
            at = at - 1 if chain else int(parents[at])
        got.append(path)
    return got


def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers
    st = prepare(case, seed)
    S = st["S"]
    off = _offsets(_counts(case))
    parents = st["parents"].cpu().numpy() if st.get("parents") is not None else None
    if case["op"] == "append":
        page, slots, ctx = st["page"], st["slots"].cpu().numpy(), st["ctx_len"].cpu().numpy()
        src, dst = st["copy_src"].cpu().numpy(), st["copy_dst"].cpu().numpy()
        k, v = st["k_cache"].double(), st["v_cache"].double()
        for s in range(S):
            if src[s] >= 0:
                part = int(ctx[s]) % page
                k[int(dst[s]), :, :part] = k[int(src[s]), :, :part].clone()
                v[int(dst[s]), :, :part] = v[int(src[s]), :, :part].clone()
        at, to = torch.from_numpy(slots // page).to(DEV), torch.from_numpy(slots % page).to(DEV)
        k[at, :, to], v[at, :, to] = st["kv"][:, 0].double(), st["kv"][:, 1].double()
        return dict(k_cache=k, v_cache=v)
    if case["op"] == "attn":
        Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], st["page"]
        g = Hq // Hkv
        out = torch.empty(st["R"], Hq, D, dtype=torch.float64, device=DEV)
        lse = torch.empty(st["R"], Hq, dtype=torch.float64, device=DEV)
        ctx, table = st["ctx_len"].cpu().numpy(), st["table"].long()
        for s in range(S):
            a, n, c = int(off[s]), int(off[s + 1] - off[s]), int(ctx[s])
            ids = table[s, : (c + n + page - 1) // page]
            K = st["k_cache"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, : c + n].double()
            V = st["v_cache"][ids].transpose(0, 1).reshape(Hkv, -1, D)[:, : c + n].double()
            hide = torch.zeros(n, c + n, dtype=torch.bool)
            hide[:, c:] = True
            for t, path in enumerate(_paths(None if parents is None else parents[a: a + n], n, parents is None)):
                hide[t, [c + j for j in path]] = False
            q = st["q"][a: a + n].double().reshape(n, Hkv, g, D)
            z = torch.einsum("thgd,hld->thgl", q, K) * st["scale"]
            z = z.masked_fill(hide.to(DEV)[:, None, None], NEG)
            lse[a: a + n] = torch.logsumexp(z, -1).reshape(n, Hq)
            out[a: a + n] = torch.einsum("thgl,hld->thgd", torch.softmax(z, -1), V).reshape(n, Hq, D)
        return dict(out=out, lse=lse)
    V = case["V"]
    out = st["logits"].double()
    ho, ht, nt = st["hist_offsets"].cpu().numpy(), st["hist_tokens"].cpu().numpy(), st["node_tokens"].cpu().numpy()
    bo, bt, bv = (st[k].cpu().numpy() for k in ("bias_offsets", "bias_tokens", "bias_values"))
    rep, pres, freq = (st[k].cpu().numpy().astype(np.float64) for k in ("repetition", "presence", "frequency"))
    for s in range(S):
        a, n = int(off[s]), int(off[s + 1] - off[s])
        base = np.bincount(ht[ho[s]: ho[s + 1]], minlength=V)
        for t, path in enumerate(_paths(None if parents is None else parents[a: a + n], n, parents is None)):
            count = base.copy()
            np.add.at(count, nt[[a + j for j in path]], 1)
            at = np.nonzero(count)[0]
            z = out[a + t, torch.from_numpy(at).to(DEV)].cpu().numpy()
            z = np.where(z > 0, z / rep[s], z * rep[s]) - freq[s] * count[at] - pres[s]
            out[a + t, torch.from_numpy(at).to(DEV)] = torch.from_numpy(z).to(DEV)
            b = torch.from_numpy(bt[bo[s]: bo[s + 1]].astype(np.int64)).to(DEV)
            out[a + t, b] += torch.from_numpy(bv[bo[s]: bo[s + 1]].astype(np.float64)).to(DEV)
    if st["allowed"] is not None:
        words = st["allowed"].cpu().numpy().view(np.uint32)
        for r in range(words.shape[0]):
            bits = np.unpackbits(words[r].astype("<u4").view(np.uint8), bitorder="little")[:V]
            out[r, torch.from_numpy(np.nonzero(bits == 0)[0]).to(DEV)] = NEG
    return dict(out=out)
