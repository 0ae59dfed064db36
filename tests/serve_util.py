"""Plain float64 forms of the operators around the verify, one sequence and one row at a time, and
builders of small inputs for their tests."""
import numpy as np

NEG = float("-inf")


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def random_parents(counts, rng):
    out = []
    for n in counts:
        out += [int(rng.integers(-1, t)) if t else -1 for t in range(n)]
    return np.array(out, np.int32)


def seen_lists(counts, parents=None, mask=None):
    """For every row the sorted list of the nodes of its own sequence that it sees."""
    got, a = [], 0
    for n in counts:
        for t in range(n):
            if mask is not None:
                got.append([j for j in range(n) if (int(mask[a + t, j // 32]) >> (j % 32)) & 1])
            elif parents is None:
                got.append(list(range(t + 1)))
            else:
                path, at = [], t
                while at >= 0:
                    path.append(at)
                    at = int(parents[a + at])
                got.append(sorted(path))
        a += n
    return got


def mask_words(counts, T, lists):
    words = np.zeros((sum(counts), (T + 31) // 32), np.uint32)
    for r, path in enumerate(lists):
        for j in path:
            words[r, j // 32] |= np.uint32(1 << (j % 32))
    return words


def slot_map(ctx, counts, table, refcount, page):
    """The rule of kv_slot_map as it is written down: sequences and pages in order."""
    table, ref0 = table.copy(), refcount
    ref = refcount.copy()
    free = iter(np.nonzero(ref0 == 0)[0])
    src, dst = np.full(len(ctx), -1, np.int32), np.full(len(ctx), -1, np.int32)
    slots = []
    for s, (c, n) in enumerate(zip(ctx, counts)):
        c, n = int(c), int(n)
        if n:
            for j in range(c // page, (c + n + page - 1) // page):
                old = int(table[s, j])
                if old >= 0 and ref0[old] <= 1:
                    continue
                new = int(next(free))
                table[s, j] = new
                ref[new] = 1
                if old >= 0:
                    ref[old] -= 1
                    if j == c // page and c % page:
                        src[s], dst[s] = old, new
        slots += [int(table[s, (c + i) // page]) * page + (c + i) % page for i in range(n)]
    return dict(table_out=table, refcount_out=ref, slots=np.array(slots, np.int64), copy_src=src, copy_dst=dst)


def attention(q, k_cache, v_cache, table, ctx, counts, lists, scale):
    """q [R, Hq, D], caches [pages, Hkv, page, D] in float64. Returns out, lse and, for error bounds,
    sum_x p_x |V_x| and the largest sum_d |q_d k_d| of each row and head."""
    R, Hq, D = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    g = Hq // Hkv
    out, lse = np.zeros((R, Hq, D)), np.full((R, Hq), NEG)
    spread, reach = np.zeros((R, Hq, D)), np.zeros((R, Hq))
    r = 0
    for s, n in enumerate(counts):
        c = int(ctx[s])
        for t in range(n):
            pos = np.concatenate([np.arange(c), c + np.array(lists[r], np.int64)]).astype(np.int64)
            if pos.size:
                ids = table[s, pos // page]
                K, V = k_cache[ids, :, pos % page], v_cache[ids, :, pos % page]  # [keys, Hkv, D]
                for h in range(Hq):
                    k, v = K[:, h // g], V[:, h // g]
                    z = (k @ q[r, h]) * scale
                    m = z.max()
                    e = np.exp(z - m)
                    p = e / e.sum()
                    out[r, h] = p @ v
                    lse[r, h] = m + np.log(e.sum())
                    spread[r, h] = p @ np.abs(v)
                    reach[r, h] = (np.abs(k) @ np.abs(q[r, h])).max() * abs(scale)
            r += 1
    return out, lse, spread, reach


def attention_bounds(spread, reach, out, D, keys, bf16):
    """How far a float32 (or bf16 in and out) evaluation may be from the exact one.

    A score is a sum of D float32 products times a constant: off by at most (D + 3) 2^-24 reach, and its
    weight by that relative amount plus 2^-22 for the exponential and its argument's rounding (the
    argument is at most 2 reach log2(e) below zero, rounded to 2^-24 of itself). Sums of `keys` weights
    and products add keys 2^-24, in any order and in pieces. The division cancels nothing: numerator and
    denominator are each off by that, so twice it, relative to sum p |v|. In bf16 (8 significant bits: a
    rounding is off by at most 2^-8 of the value, reached just above a power of two) each weight is further
    rounded for the product with V, and so is the result."""
    eps = 2.0 ** -24
    rel = (D + 3) * eps * reach + 4 * eps + 4 * reach * eps
    tot = 2 * (rel + (keys + 8) * eps)
    b = tot[..., None] * spread
    if bf16:
        u = 2.0 ** -8
        b = b + u * spread
        b = b + u * (np.abs(out) + b)
    return b + 1e-30, tot


def process_logits(logits, counts, lists, V, node_tokens=None, hist=None, repetition=None, presence=None,
                   frequency=None, bias=None, allowed=None):
    """hist: a list of tokens for each sequence; bias: a list of (token, value) for each."""
    z = logits.astype(np.float64).copy()
    r = a = 0
    for s, n in enumerate(counts):
        for t in range(n):
            count = np.zeros(V)
            for tok in (hist[s] if hist is not None else []):
                if tok >= 0:
                    count[tok] += 1
            if node_tokens is not None:
                for j in lists[r]:
                    if node_tokens[a + j] >= 0:
                        count[node_tokens[a + j]] += 1
            hit = count > 0
            rep = 1.0 if repetition is None else float(repetition[s])
            x = z[r]
            with np.errstate(invalid="ignore"):
                x = np.where(hit, np.where(x > 0, x / rep, x * rep), x)
                if frequency is not None:
                    x = np.where(hit, x - float(frequency[s]) * count, x)
                if presence is not None:
                    x = np.where(hit, x - float(presence[s]), x)
            for tok, val in {tok: val for tok, val in (bias[s] if bias is not None else [])}.items():
                if tok >= 0:
                    x[tok] += float(val)
            if allowed is not None:
                bits = np.unpackbits(allowed[r].astype("<u4").view(np.uint8), bitorder="little")[:V]
                x = np.where(bits != 0, x, NEG)
            z[r] = x
            r += 1
        a += n
    return z
