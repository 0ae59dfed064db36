"""Beam search over a paged cache, whole on the device: a toy target (one attention layer, random) and G prompts with N beams each.

A step:
  kv_slot_map         the page and slot of each beam's new token, with copies of pages that beams share
  kv_append           its key and value
  tree_attention      the new token over the cache; the pages that a prompt's beams share are read once
  beam_select         the N best continuations of each prompt's beams; finished beams stay as they are
  state_reorder       the beams' tokens follow their ancestors, and so do
  kv_pagetable_remap  their page tables
Around it: kv_fork gives the pages of a prompt to its beams, kv_free lets go of those of prompts that have ended, kv_compact and
kv_copy_pages move the pages that are still in use to the front of the cache.

    python examples/beam_search.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from smc_reweight_resample_gb300 import _binding as lib  # noqa: E402


class Search:
    def __init__(self, G=3, N=4, V=1024, Hq=4, Hkv=2, D=64, page=16, pages_per_seq=12, prompt=(40, 17, 64), eos=0, seed=0, dtype=torch.float32):
        self.G, self.N, self.V, self.Hq, self.Hkv, self.D, self.page, self.P, self.eos = G, N, V, Hq, Hkv, D, page, pages_per_seq, eos
        self.S, self.num_pages = G * N, 2 * G * N * pages_per_seq
        gen, dev, S, width = torch.Generator("cuda").manual_seed(seed), "cuda", self.S, 128

        def random(*shape, scale):
            return (torch.randn(*shape, device=dev, generator=gen) * scale).to(dtype)

        self.embed = random(V, width, scale=1.0)
        # queries, keys and values depend on the token alone: one row of this table for each
        self.qkv = self.embed @ random(width, (Hq + 2 * Hkv) * D, scale=width ** -0.5)
        self.w_out, self.head = random(Hq * D, width, scale=(Hq * D) ** -0.5), random(width, V, scale=width ** -0.5)
        # the cache as a list of layers' keys and values, as kv_copy_pages takes it
        self.caches = [torch.zeros(self.num_pages, Hkv, page, D, device=dev, dtype=dtype) for _ in range(2)]

        self.ws_slots = lib.Workspace(lib.OP_KV_SLOT_MAP, S, 0, self.num_pages)
        self.ws_append = lib.Workspace(lib.OP_KV_APPEND, S)
        self.ws_attn = lib.TreeAttentionWorkspace(S, N, 1, Hq, Hkv, D)
        self.ws_select = lib.Workspace(lib.OP_BEAM_SELECT, S, 0, V)
        self.ws_pages = lib.Workspace(lib.OP_KV_COMPACT, S, 0, self.num_pages)
        self.ws_remap = lib.Workspace(lib.OP_PAGETABLE_REMAP, G)

        # prompts: the first beam of each takes all tokens but the last, then its pages are forked
        lengths = torch.tensor([prompt[g % len(prompt)] for g in range(G)], device=dev)
        self.tokens = torch.full((S, pages_per_seq * page + 1), -1, dtype=torch.int32, device=dev)  # -1: none yet
        for g in range(G):
            n = int(lengths[g])
            self.tokens[g * N:(g + 1) * N, :n] = torch.randint(1, V, (n,), device=dev, generator=gen, dtype=torch.int32)
        new = torch.zeros(S, dtype=torch.int64, device=dev)
        new[::N] = lengths - 1
        offsets = torch.cat([new.new_zeros(1), new.cumsum(0)]).to(torch.int32)
        table = torch.full((S, pages_per_seq), -1, dtype=torch.int32, device=dev)
        refcount = torch.zeros(self.num_pages, dtype=torch.int32, device=dev)
        self.ctx = torch.zeros(S, dtype=torch.int32, device=dev)
        got = lib.kv_slot_map(self.ctx, table, refcount, S, int(new.max()), page, new_offsets=offsets, rows=int(offsets[-1]), ws=self.ws_slots)
        self.append(torch.cat([self.tokens[s, :int(new[s])] for s in range(0, S, N)]), got)
        first = torch.arange(S, device=dev, dtype=torch.int32) // N * N
        self.table, self.refcount = lib.kv_fork(got["table_out"], got["refcount_out"], first, page, ws=self.ws_pages)
        self.ctx = (lengths - 1).repeat_interleave(N).to(torch.int32)
        # one beam of each prompt to begin with
        self.scores = torch.full((G, N), float("-inf"), device=dev)
        self.scores[:, 0] = 0
        self.scores, self.finished = self.scores.flatten(), torch.zeros(S, dtype=torch.int32, device=dev)

    def append(self, tokens, slots):
        """Keys and values of the new tokens into the cache; returns the queries."""
        q, k, v = self.qkv[tokens.long()].split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], dim=1)
        lib.kv_append(k.unflatten(1, (self.Hkv, self.D)), v.unflatten(1, (self.Hkv, self.D)), slots["slots"], *self.caches, ctx_len=self.ctx,
                      copy_src=slots["copy_src"], copy_dst=slots["copy_dst"], ws=self.ws_append)
        return q.unflatten(1, (self.Hq, self.D))

    def step(self):
        S, N, G = self.S, self.N, self.G
        last = self.tokens.gather(1, self.ctx[:, None].long())[:, 0]
        slots = lib.kv_slot_map(self.ctx, self.table, self.refcount, S, 1, self.page, ws=self.ws_slots)
        q = self.append(last, slots)
        o, _ = lib.tree_attention(q, *self.caches, slots["table_out"], self.ctx, S, 1, self.D ** -0.5, N=N, ws=self.ws_attn, with_lse=False)
        logits = (self.embed[last.long()] + o.flatten(1) @ self.w_out) @ self.head
        got = lib.beam_select(logits, G, N, self.V, N, scores=self.scores, finished=self.finished, pad_token=self.eos, eos_token=self.eos,
                              ws=self.ws_select)
        (self.tokens,) = lib.state_reorder([self.tokens], got["ancestors"], G, N, ws=self.ws_pages)
        self.table, self.refcount = lib.kv_pagetable_remap(got["ancestors"], None, G, N, slots["table_out"], self.P, self.num_pages, ws=self.ws_remap)
        self.ctx = self.ctx + 1  # alike in all beams of a prompt
        self.tokens.scatter_(1, self.ctx[:, None].long(), got["tokens"][:, None])
        self.scores, self.finished = got["scores"], got["finished"]
        return got

    def release(self, groups):
        """Lets go of the pages of the prompts `groups` and moves the others' to the front. Returns how many are in use."""
        keep = torch.full((self.G, self.N), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        keep[groups] = 0
        table, refcount = lib.kv_free(self.table, self.refcount, keep.flatten(), self.page, ws=self.ws_pages)
        got = lib.kv_compact(table, refcount, ws=self.ws_pages)
        lib.kv_copy_pages(self.caches, got["src"], got["dst"], count=got["counts"], ws=self.ws_pages)
        self.table, self.refcount = got["table_out"], got["refcount_out"]
        return got["counts"][1]

    def check(self):
        for ws in (self.ws_slots, self.ws_append, self.ws_attn, self.ws_select, self.ws_pages, self.ws_remap):
            if (status := lib.check_status(ws)) != 0:
                raise lib.SMCSDError(status, "search")


def main(steps=20):
    search = Search()
    start = search.ctx.clone()
    for _ in range(steps):
        search.step()
    search.check()
    for g in range(search.G):
        for n in range(search.N):
            s = g * search.N + n
            print(f"prompt {g}: {float(search.scores[s]):8.3f}  {search.tokens[s, int(start[s]) + 1:int(search.ctx[s]) + 1].tolist()}")
    held = int((search.refcount > 0).sum())
    print(f"{held} pages in use; without prompt 0 {int(search.release([0]))}")
    search.check()


if __name__ == "__main__":
    main()
