"""A draft's head learns the target's distribution from the target's top logits: what a speculative decoder gains acceptance by.

A step over R tokens:
  beam_select    (one beam a row) the target's K largest log-probabilities: the teacher's list
  distill_loss   the draft's loss against it, the rest of the vocabulary as one event, and the gradient of its logits
and the head's gradient is the hidden states' product with that.

    python examples/distill_draft.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from smc_reweight_resample_gb300 import _binding as lib  # noqa: E402


class Draft:
    def __init__(self, R=512, V=4096, width=256, K=32, temperature=1.0, seed=0, dtype=torch.float32):
        self.R, self.V, self.K, self.temperature = R, V, K, temperature
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.target_head = (torch.randn(width, V, device="cuda", generator=self.gen) * 3 * width ** -0.5).to(dtype)
        self.head = (torch.randn(width, V, device="cuda", generator=self.gen) * width ** -0.5).to(dtype)
        self.ws_top = lib.Workspace(lib.OP_BEAM_SELECT, R, 0, V)
        self.ws_loss = lib.Workspace(lib.OP_DISTILL_LOSS, R)

    def hidden(self):
        return torch.randn(self.R, self.head.shape[0], device="cuda", generator=self.gen).to(self.head.dtype)

    def teacher(self, hidden):
        top = lib.beam_select(hidden @ self.target_head, self.R, 1, self.V, self.K, temperature=self.temperature, ws=self.ws_top)
        return top["tokens"].view(self.R, self.K), top["scores"].view(self.R, self.K)

    def gradient(self, hidden, tokens, values, weight):
        """The rows' losses and the head's gradient of their sum with these weights."""
        logits = hidden @ self.head
        loss, dlogits = lib.distill_loss(logits, tokens, values, self.V, temperature=self.temperature, rest=True, weight=weight, dlogits=logits,
                                         ws=self.ws_loss)
        return loss, hidden.t() @ dlogits

    def step(self, rate=20.0):
        hidden = self.hidden()
        weight = torch.full((self.R,), 1.0 / self.R, device="cuda")
        loss, grad = self.gradient(hidden, *self.teacher(hidden), weight)
        self.head -= rate * grad
        return loss

    def check(self):
        for ws in (self.ws_top, self.ws_loss):
            if (status := lib.check_status(ws)) != 0:
                raise lib.SMCSDError(status, "distillation")


def main(steps=20):
    draft = Draft()
    for i in range(steps):
        loss = draft.step()
        draft.check()
        print(f"step {i}: loss {float(loss.mean()):.4f}")


if __name__ == "__main__":
    main()
