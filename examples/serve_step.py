"""Speculative decoding by sequential Monte Carlo, whole steps on the device: a toy target (one attention
layer) and a toy draft (it looks at the last token only), both random, over a paged cache.

A step of G prompts with N particles each and K drafts:
  draft_sample    K draft tokens of every particle, with their log q
  kv_slot_map     pages and slots of the K+1 new tokens, with copies of pages that particles share
  kv_append       their keys and values
  tree_attention  the new tokens over the cache; the pages that a prompt's particles share are read once
  logits_process  the repetition penalty, over each particle's own tokens
  smc_step_logq   weights, the (K+1)-th token, resampling, and the particles' pages after it

    python examples/serve_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from smc_reweight_resample_gb300 import _binding as lib  # noqa: E402


class Session:
    def __init__(self, G=4, N=8, K=4, V=2048, Hq=8, Hkv=2, D=64, page=16, pages_per_seq=16, prompt=(70, 33, 90, 1), seed=0,
                 dtype=torch.bfloat16):
        self.G, self.N, self.K, self.V, self.Hq, self.Hkv, self.D, self.page = G, N, K, V, Hq, Hkv, D, page
        self.S, self.T, self.P = G * N, K + 1, pages_per_seq
        self.num_pages = self.S * pages_per_seq
        self.gen = torch.Generator("cuda").manual_seed(seed)
        dev, S, T, width = "cuda", self.S, self.T, 256

        def random(*shape, scale):
            return (torch.randn(*shape, device=dev, generator=self.gen) * scale).to(dtype)

        embed = random(V, width, scale=1.0)
        # queries, keys and values depend on the token alone: one row of this table for each
        self.qkv = embed @ random(width, (Hq + 2 * Hkv) * D, scale=width ** -0.5)
        self.embed, self.w_out = embed, random(Hq * D, width, scale=(Hq * D) ** -0.5)
        self.head, self.draft_head = random(width, V, scale=0.5 * width ** -0.5), random(width, V, scale=0.5 * width ** -0.5)
        self.k_cache = torch.zeros(self.num_pages, Hkv, page, D, device=dev, dtype=dtype)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.logw = torch.zeros(S, device=dev)
        self.repetition = torch.full((S,), 1.2, device=dev)

        self.ws_draft = lib.Workspace(lib.OP_DRAFT_SAMPLE, S, 0, V)
        self.ws_slots = lib.Workspace(lib.OP_KV_SLOT_MAP, S, 0, self.num_pages)
        self.ws_append = lib.Workspace(lib.OP_KV_APPEND, S)
        self.ws_attn = lib.TreeAttentionWorkspace(S, N, T, Hq, Hkv, D)
        self.ws_logits = lib.Workspace(lib.OP_LOGITS_PROCESS, S)
        self.ws_step = lib.Workspace(lib.OP_SMC_STEP, S, K, V)

        # prompts: the first particle of each takes all tokens but the last, then all of its prompt's particles hold its pages
        lengths = torch.tensor([prompt[g % len(prompt)] for g in range(G)], device=dev)
        self.tokens = torch.full((S, pages_per_seq * page + 1), -1, dtype=torch.int32, device=dev)  # -1: none yet
        for g in range(G):
            n = int(lengths[g])
            self.tokens[g * N:(g + 1) * N, :n] = torch.randint(V, (n,), device=dev, generator=self.gen, dtype=torch.int32)
        self.hist_offsets = torch.arange(S + 1, device=dev, dtype=torch.int32) * self.tokens.shape[1]
        new = torch.zeros(S, dtype=torch.int64, device=dev)
        new[::N] = lengths - 1
        offsets = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
        table = torch.full((S, pages_per_seq), -1, dtype=torch.int32, device=dev)
        refcount = torch.zeros(self.num_pages, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(S, dtype=torch.int32, device=dev)
        rows = int(offsets[-1])
        if rows:
            got = lib.kv_slot_map(self.ctx, table, refcount, S, int(new.max()), page, new_offsets=offsets, rows=rows, ws=self.ws_slots)
            self.append(torch.cat([self.tokens[s, :int(new[s])] for s in range(0, S, N)]), got)
            table, refcount = lib.kv_pagetable_remap(torch.zeros(S, dtype=torch.int32, device=dev),
                                                     torch.ones(G, dtype=torch.int32, device=dev), G, N, got["table_out"],
                                                     pages_per_seq, self.num_pages)
        self.table, self.refcount = table, refcount
        self.ctx = (lengths - 1).repeat_interleave(N).to(torch.int32)

    def uniform(self, *shape):
        return torch.rand(*shape, device="cuda", generator=self.gen)

    def append(self, tokens, slots):
        """Keys and values of the new tokens (slices of their projections) into the cache; returns the queries."""
        q, k, v = self.qkv[tokens.long()].split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1)
        lib.kv_append(k.unflatten(1, (self.Hkv, self.D)), v.unflatten(1, (self.Hkv, self.D)), slots["slots"], self.k_cache, self.v_cache,
                      ctx_len=self.ctx, copy_src=slots["copy_src"], copy_dst=slots["copy_dst"], ws=self.ws_append)
        return q.unflatten(1, (self.Hq, self.D))

    def step(self, temperature=1.0, alpha=1.0):
        S, K, T, V, G, N = self.S, self.K, self.T, self.V, self.G, self.N
        ess_threshold = N / 2
        last = self.tokens.gather(1, self.ctx[:, None].long())[:, 0]
        nodes, logq = [last], []
        for _ in range(K):
            logits = self.embed[nodes[-1].long()] @ self.draft_head
            token, lq = lib.draft_sample(logits, S, V, temperature, self.uniform(S), ws=self.ws_draft)
            nodes.append(token)
            logq.append(lq)
        nodes, logq = torch.stack(nodes, 1), torch.stack(logq, 1)

        slots = lib.kv_slot_map(self.ctx, self.table, self.refcount, S, T, self.page, ws=self.ws_slots)
        q = self.append(nodes.flatten(), slots)
        o, _ = lib.tree_attention(q, self.k_cache, self.v_cache, slots["table_out"], self.ctx, S, T, self.D ** -0.5, N=N,
                                  ws=self.ws_attn, with_lse=False)
        logits = (self.embed[nodes.flatten().long()] + o.flatten(1) @ self.w_out) @ self.head
        lib.logits_process(logits, S, T, V, node_tokens=nodes.flatten(), hist_tokens=self.tokens.flatten(),
                           hist_offsets=self.hist_offsets, repetition=self.repetition, out=logits, ws=self.ws_logits)
        got = lib.smc_step_logq(logits, nodes[:, 1:].contiguous(), logq.contiguous(), G, N, K, V, temperature, alpha, self.uniform(S),
                                self.logw, ess_threshold, self.uniform(G), table_in=slots["table_out"], pages_per_seq=self.P,
                                num_pages=self.num_pages, ws=self.ws_step)

        new = torch.cat([nodes[:, 1:], got["bonus_token"][:, None]], 1)
        at = self.ctx[:, None].long() + 1 + torch.arange(T, device="cuda")
        self.tokens.scatter_(1, at, new)
        parent = torch.arange(S, device="cuda") // N * N + got["ancestors"].long()
        self.tokens = self.tokens[parent]
        self.ctx = self.ctx + T  # alike in all particles of a prompt
        self.table, self.refcount = got["table_out"], got["refcount"]
        return got

    def check(self):
        for ws in (self.ws_draft, self.ws_slots, self.ws_append, self.ws_attn, self.ws_logits, self.ws_step):
            if (status := lib.check_status(ws)) != 0:
                raise lib.SMCSDError(status, "step")


def main(steps=8):
    session = Session()
    start = session.ctx.clone()
    for i in range(steps):
        got = session.step()
        session.check()
        held = int((session.refcount > 0).sum())
        print(f"step {i}: ESS {[round(x, 2) for x in got['ess'].tolist()]}, resampled {got['resampled'].tolist()}, "
              f"{held} pages held for {int((session.table >= 0).sum())} table entries")
    for g in range(session.G):
        s = g * session.N
        print(f"prompt {g}: {session.tokens[s, int(start[s]) + 1:int(session.ctx[s]) + 1].tolist()}")


if __name__ == "__main__":
    main()
