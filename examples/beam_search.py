"""Beam search over a paged cache: several requests at once, their beams' pages shared until
they are written.

    python examples/beam_search.py

One attention layer stands for the model (its projections are tables of random rows, one
per token), so that what this library does in a step is all there is to see: room for the
new rows, the copies of shared pages, the append, the attention, the choice of the next
tokens, and the sequences reordered by it.  Nothing is read back between the steps.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_expert_weight_gb300.smoe as S  # noqa: E402


class TinyModel:
    """One attention layer between an embedding and a head, all random."""

    def __init__(self, vocab, heads, kv_heads, head_dim, device, seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device).bfloat16()

        self.heads, self.kv_heads, self.vocab = heads, kv_heads, vocab
        self.qkv = randn(vocab, heads + 2 * kv_heads, head_dim)
        self.head = randn(heads * head_dim, vocab)

    def project(self, tokens):
        return self.qkv[tokens.long()].split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def logits(self, a):
        return a.flatten(1) @ self.head


class BeamSearch:
    """The beams of several requests; sequence g * beams + k is beam k of request g."""

    def __init__(self, model, requests, beams, num_pages, page, max_pages, head_dim, end_token,
                 device):
        self.model, self.beams, self.end, self.page = model, beams, end_token, page
        n, i32 = requests * beams, dict(dtype=torch.int32, device=device)
        pool = torch.zeros(num_pages, 2, model.kv_heads, page, head_dim, dtype=torch.bfloat16,
                           device=device)
        self.k_pages, self.v_pages = pool[:, 0], pool[:, 1]
        self.refs, self.kv_len = torch.zeros(num_pages, **i32), torch.zeros(n, **i32)
        self.table = torch.zeros(n, max_pages, **i32)
        self.copies, self.counts = torch.zeros(n, 2, **i32), torch.zeros(2, **i32)
        self.single = torch.arange(n + 1, **i32)      # row starts of a step of one row each
        # the first choice is made among the continuations of each request's first beam
        self.scores = torch.full((requests, beams), float("-inf"), device=device)
        self.scores[:, 0] = 0
        self.tokens = torch.full((requests, beams), -1, **i32)
        self.parents = torch.zeros(requests, beams, **i32)
        self.attn_ws, self.beam_ws = S.attention_workspace(device), S.beam_workspace(device)

    @property
    def pool(self):
        return self.refs, self.kv_len, self.table, self.page

    def attend(self, tokens, row_start, max_rows):
        """The attention's output of new rows of the given tokens."""
        S.pages_reserve(*self.pool, row_start, self.copies, self.counts)
        S.pages_copy(self.k_pages, self.v_pages, self.copies, self.counts)
        where = (self.k_pages, self.v_pages, row_start, self.kv_len, self.table)
        q, k, v = self.model.project(tokens)
        q = S.kv_append(q, k, v, *where)
        return S.attention(q, *where, max_rows, self.attn_ws)

    def choose(self, logits):
        S.beam_select(logits, self.scores, self.beams, self.beam_ws, last=self.tokens,
                      end_token=self.end, out=(self.scores, self.parents, self.tokens))
        S.pages_fork(*self.pool, self.parents.view(-1))

    def prompts(self, prompts):
        """The requests' prompts (lists of tokens), each into its first beam."""
        device, start = self.refs.device, [0]
        for p in prompts:
            start += [start[-1] + len(p)] * self.beams
        start = torch.tensor(start, dtype=torch.int32).to(device)
        tokens = torch.tensor([t for p in prompts for t in p]).to(device)
        a = self.attend(tokens, start, max(len(p) for p in prompts))
        logits = self.model.logits(a[start[1::self.beams].long() - 1])
        # (the other beams have no score yet: their rows of the logits are not read)
        self.choose(logits.repeat_interleave(self.beams, 0))

    def step(self):
        """One more token of every beam.  (A beam that leads nowhere has token -1; any other
        may stand for it, its score stays -inf.  A finished one gets a row as well, which
        nothing reads: steps are alike then, and its pages go on growing with the others'.)"""
        a = self.attend(self.tokens.view(-1).clamp_min(0), self.single, 1)
        self.choose(self.model.logits(a))


def main():
    device = torch.device("cuda:0")
    model = TinyModel(500, 8, 2, 64, device)
    search = BeamSearch(model, requests=3, beams=4, num_pages=200, page=16, max_pages=20,
                        head_dim=64, end_token=2, device=device)
    g = torch.Generator().manual_seed(1)
    search.prompts([torch.randint(3, 500, (n,), generator=g).tolist() for n in (100, 33, 7)])
    history = []
    for _ in range(12):
        history.append((search.parents.clone(), search.tokens.clone()))
        search.step()
    history.append((search.parents.clone(), search.tokens.clone()))
    if S.device_status() != 0:
        raise RuntimeError("a kernel recorded a fault")
    # the best beam of each request, from its last token back to its first
    for r in range(3):
        at, said = 0, []
        for parents, tokens in reversed(history):
            said.append(int(tokens[r, at]))
            at = int(parents[r, at]) - r * search.beams
        print(f"request {r}: score {float(search.scores[r, 0]):.3f}, tokens {said[::-1]}")
    held = int((search.refs > 0).sum())
    print(f"done: {held} pages held, {int(search.refs.sum())} times")


if __name__ == "__main__":
    main()
