"""One decoder layer from this library's operators: a paged cache served to
several sequences at once, prompts in chunks beside the next tokens of others.

    python examples/decoder_layer.py

Between the norms and projections (plain torch) a step is kv_append and
attention on the paged cache and the expert layer's forward, with the sequences'
lengths and pages on the device.  Weights
are random; the layer is the synthetic generator's smallest workload.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_expert_weight_gb300.smoe as S  # noqa: E402
from bit_expert_weight_gb300 import synth as Y  # noqa: E402

EPS = 1e-6


class PagedCache:
    """One layer's keys and values, side by side in a page, and which pages each sequence
    owns.  The host keeps the free list; the device gets lengths and page ids."""

    def __init__(self, num_pages, page, kv_heads, head_dim, max_seqs, max_pages, device):
        self.page = page
        pool = torch.zeros(num_pages, 2, kv_heads, page, head_dim, dtype=torch.bfloat16,
                           device=device)
        self.k_pages, self.v_pages = pool[:, 0], pool[:, 1]
        self.free = list(range(num_pages))
        self.owned = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs
        self.table = torch.zeros(max_seqs, max_pages, dtype=torch.int32)
        self.device = device

    def grow(self, rows):
        """Make room for rows[b] more keys of every sequence; the step's (row_start, kv_len,
        page_table) on the device."""
        start = [0]
        for b, r in enumerate(rows):
            self.lens[b] += r
            while len(self.owned[b]) * self.page < self.lens[b]:
                self.table[b, len(self.owned[b])] = self.free[-1]
                self.owned[b].append(self.free.pop())
            start.append(start[-1] + r)
        i32 = torch.int32
        return (torch.tensor(start, dtype=i32).to(self.device),
                torch.tensor(self.lens, dtype=i32).to(self.device), self.table.to(self.device))

    def drop(self, b):
        """The sequence is done: its pages are free again."""
        self.free += self.owned[b]
        self.owned[b], self.lens[b] = [], 0


def rms_norm(x, weight):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()).bfloat16()


class DecoderLayer:
    def __init__(self, wl, heads, kv_heads, head_dim, device, bits=4, seed=0):
        self.wl, self.heads, self.kv_heads, self.head_dim = wl, heads, kv_heads, head_dim
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(rows, cols, gain):
            w = torch.randn(rows, cols, generator=g, device=device) * gain * cols ** -0.5
            return w.to(torch.bfloat16)

        self.w_qkv = randn((heads + 2 * kv_heads) * head_dim, wl.d, 1.0)
        self.w_out = randn(wl.d, heads * head_dim, 1.0)
        self.q_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).bfloat16()
        self.attn_norm = (1 + 0.1 * torch.randn(wl.d, generator=g, device=device)).bfloat16()
        self.experts_norm = (1 + 0.1 * torch.randn(wl.d, generator=g, device=device)).bfloat16()
        self.rope, self.rot_scale = S.rope_table(head_dim, 1e6, "parts", 4.0, device=device)
        codes, scales = [], []
        for e in range(wl.E):
            for role in (Y.ROLE_GATE, Y.ROLE_UP, Y.ROLE_DOWN):
                w = torch.from_numpy(wl.expert_weight(0, e, role).view("int16"))
                c, s = S.quantize(w.to(device).view(torch.bfloat16), bits)
                codes.append(c)
                scales.append(s)
        tiles = S.repack(codes, scales, wl.d, wl.f, wl.E, bits)
        router = torch.from_numpy(wl.router_weight(0).view("int16")).to(device)
        self.experts = S.MoELayer(wl.d, wl.f, wl.E, wl.k, wl.norm, bits,
                                  router.view(torch.bfloat16), tiles)
        self.attn_ws = S.attention_workspace(device)
        self.moe_ws = {}

    def project(self, x):
        """q, k and v of the rows, as views of one product."""
        qkv = (x @ self.w_qkv.T).view(x.shape[0], -1, self.head_dim)
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def __call__(self, x, cache, batch, max_rows):
        """x bf16 [rows, d]; batch: what cache.grow returned for these rows."""
        where = (cache.k_pages, cache.v_pages, *batch)
        q, k, v = self.project(rms_norm(x, self.attn_norm))
        q = S.kv_append(q, k, v, *where, self.rope, self.rot_scale, q_norm=self.q_norm,
                        k_norm=self.k_norm, eps=EPS)
        a = S.attention(q, *where, max_rows, self.attn_ws)
        h = x + a.flatten(1) @ self.w_out.T
        return (h + self.moe(rms_norm(h, self.experts_norm))).to(torch.bfloat16)

    def moe(self, x):
        """The experts' output of the rows.  A workspace is laid out for its number of rows, so
        the rows are filled up to a power of two: a few workspaces serve every step."""
        T = x.shape[0]
        rows = 1 << max(0, T - 1).bit_length()
        if rows not in self.moe_ws:
            self.moe_ws[rows] = S.workspace(self.experts, rows)
        x = torch.nn.functional.pad(x, (0, 0, 0, rows - T))
        return S.forward(self.experts, x, self.moe_ws[rows])[:T]


def main():
    device = torch.device("cuda:0")
    wl = Y.WORKLOADS["tiny"]
    layer = DecoderLayer(wl, heads=8, kv_heads=2, head_dim=64, device=device)
    prompts, chunk, new_tokens = [300, 37, 1, 120], 64, 5
    cache = PagedCache(64, 16, 2, 64, len(prompts), 32, device)
    g = torch.Generator(device=device)
    g.manual_seed(1)
    left, made, last = list(prompts), [0] * len(prompts), [None] * len(prompts)
    step = 0
    while any(m < new_tokens for m in made):
        # a chunk of what is left of each prompt, beside the next token of the others
        rows = [min(n, chunk) if n else int(m < new_tokens) for n, m in zip(left, made)]
        batch = cache.grow(rows)
        parts = []
        for b, r in enumerate(rows):
            if left[b]:
                parts.append(torch.randn(r, wl.d, generator=g, device=device).bfloat16())
            elif r:
                parts.append(last[b])
        y = layer(torch.cat(parts), cache, batch, max(rows))
        at = 0
        for b, r in enumerate(rows):
            if r:
                last[b] = y[at + r - 1:at + r]
                made[b] += int(not left[b])
                left[b] = max(0, left[b] - r)
                at += r
            if made[b] == new_tokens and cache.owned[b]:
                cache.drop(b)
        step += 1
        print(f"step {step}: rows {rows}, keys {cache.lens}, pages free {len(cache.free)}")
    if S.device_status() != 0:
        raise RuntimeError("a kernel recorded a fault")
    print("done:", made, "tokens made")


if __name__ == "__main__":
    main()
