"""Plain float64 forms of beam selection, the pages' housekeeping and the distillation loss, for their tests."""
import numpy as np
import torch

NEG = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def beam_select(logits, G, N, V, M, temperature=1.0, scores=None, finished=None, pad=0, eos=-1):
    """logits float64 [G*N, V]. Returns tokens, ancestors, scores (float64), finished, each [G, M], and the smallest difference between
    neighbours of different beams in the order that the selection depends on."""
    c = 1.0 / float(np.float32(temperature))
    tokens, anc = np.full((G, M), pad), np.zeros((G, M), int)
    out, over = np.full((G, M), NEG), np.ones((G, M), int)
    gap = np.inf
    for g in range(G):
        cand = []  # (score, beam, place) as arrays
        for i in range(N):
            s = 0.0 if scores is None else float(scores[g * N + i])
            if s == NEG:
                continue
            if finished is not None and finished[g * N + i]:
                cand.append((np.array([s]), np.array([i]), np.array([-1])))
                continue
            z = logits[g * N + i]
            if not (z > NEG).any():
                continue
            m = z.max()
            z, m = (z - m) * c, 0.0
            x = s - np.log(np.exp(z - m).sum()) + (z - m)
            cand.append((x, np.full(V, i), np.arange(V)))
        if not cand:
            continue
        x, beam, at = (np.concatenate([q[k] for q in cand]) for k in range(3))
        keep = x > NEG
        x, beam, at = x[keep], beam[keep], at[keep]
        order = np.lexsort((at, beam, -x))[:M + 1]
        x, beam, at = x[order], beam[order], at[order]
        near = np.diff(x)[np.diff(beam) != 0]
        gap = min(gap, np.abs(near).min() if near.size else np.inf)
        n = min(M, x.size)
        for m in range(n):
            b, v = int(beam[m]), int(at[m])
            tokens[g, m], anc[g, m], out[g, m] = (pad if v < 0 else v), b, x[m]
            over[g, m] = v < 0 or (eos >= 0 and v == eos)
    return tokens, anc, out, over, gap


def fork(table, refcount, parents, lengths, page):
    """Tables and counts after kv_fork's rule."""
    S, P = table.shape
    out = np.full_like(table, -1)
    for s in range(S):
        parent = s if parents is None else int(parents[s])
        if parent < 0:
            continue
        n = P if lengths is None else min(P, -(-int(lengths[s]) // page))
        out[s, :n] = table[parent, :n]
    ref = refcount + np.bincount(out[out >= 0].ravel(), minlength=refcount.size) - np.bincount(table[table >= 0].ravel(),
                                                                                               minlength=refcount.size)
    return out, ref.astype(np.int32)


def compact(table, refcount):
    used = int((refcount > 0).sum())
    dst = [i for i in range(used) if refcount[i] <= 0]
    src = [i for i in range(used, refcount.size) if refcount[i] > 0]
    to = np.arange(refcount.size)
    to[src] = dst
    out = table.copy()
    out[table >= 0] = to[table[table >= 0]]
    ref = np.zeros_like(refcount)
    for i in range(refcount.size):
        if refcount[i] > 0:
            ref[to[i]] = refcount[i]
    return out, ref, np.array(src, int), np.array(dst, int), used


def distill(z, tokens, values, V, temperature=1.0, rest=False, weight=None):
    """z float64 [R, V]. Returns loss [R], gradient [R, V] and, for error bounds, of each row: the largest |log| that enters the
    loss, sum of p, q [R, V] and the part of the gradient of unlisted tokens that p_r makes."""
    R, K = tokens.shape
    T = float(np.float32(temperature))
    loss, grad = np.zeros(R), np.zeros((R, V))
    scale, parts = np.zeros(R), np.zeros((R, V))
    for r in range(R):
        there = tokens[r] >= 0
        ids, val = tokens[r][there], values[r][there].astype(np.float64)
        if not (val > NEG).any():
            continue
        x = z[r] / T
        m = x.max()
        lse = m + np.log(np.exp(x - m).sum())
        logq = x - lse
        q = np.exp(logq)
        if rest:
            logp = val
        else:
            logp = val - (val.max() + np.log(np.exp(val - val.max()).sum()))
        p = np.exp(logp)
        p_r = max(0.0, 1.0 - p.sum()) if rest else 0.0
        P = p.sum() + p_r
        on = p > 0
        loss[r] = (p[on] * (logp[on] - logq[ids[on]])).sum()
        scale[r] = (p[on] * (1 + np.abs(logp[on]) + np.abs(x[ids[on]] - m) + abs(lse - m))).sum()
        listed = np.zeros(V, bool)
        listed[ids] = True
        d = q * P
        part = q * P
        if rest and p_r > 0:
            out = logq[~listed]
            top = out.max() if out.size else NEG
            if top > NEG:
                away = np.exp(out - top)
                logq_r, away = top + np.log(away.sum()), away / away.sum()  # the rest's own softmax, however small q_r is
                loss[r] += p_r * (np.log(p_r) - logq_r)
                # p_r itself is a difference: 1 - sum p
                scale[r] += p_r * (1 + abs(np.log(p_r)) + abs(logq_r)) + (1 + abs(np.log(p_r) - logq_r))
                d[~listed] -= p_r * away
                part[~listed] += (p_r + 1) * away
            else:
                loss[r] = np.inf
        np.subtract.at(d, ids, p)
        np.add.at(part, ids, p)
        w = 1.0 if weight is None else float(weight[r])
        grad[r] = w / T * d
        parts[r] = abs(w) / T * part
    return loss, grad, scale, parts


def as_float64(t):
    return t.detach().double().cpu().numpy()
