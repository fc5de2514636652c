"""Plain definitions of the beams' selection and of a page pool's upkeep, and the error
bound that the selection's fp32 sums allow."""
from __future__ import annotations

import math
import random

import torch

U32 = 2.0 ** -24


def pages_of(n, page):
    return -(-n // page)


class Pool:
    """A pool and its sequences on the host, one step after the other."""

    def __init__(self, num_pages, page, num_seqs, width, fill=-9):
        self.page, self.width = page, width
        self.refs, self.kv = [0] * num_pages, [0] * num_seqs
        self.table = [[fill] * width for _ in range(num_seqs)]

    def used(self, s):
        return self.table[s][:pages_of(self.kv[s], self.page)]

    def copy(self):
        p = Pool.__new__(Pool)
        p.page, p.width, p.refs, p.kv = self.page, self.width, list(self.refs), list(self.kv)
        p.table = [list(r) for r in self.table]
        return p

    def fork(self, parent, keep=None):
        was, kv = [self.used(s) for s in range(len(self.kv))], list(self.kv)
        for s, p in enumerate(parent):
            self.kv[s] = kv[p] if p >= 0 else 0
            if keep is not None:
                self.kv[s] = min(self.kv[s], max(keep[s], 0))
            n = pages_of(self.kv[s], self.page)
            if p >= 0:
                self.table[s][:n] = was[p][:n]
        for row in was:
            for p in row:
                self.refs[p] -= 1
        for s in range(len(self.kv)):
            for p in self.used(s):
                self.refs[p] += 1

    def reserve(self, rows):
        """(copies, pages left); None: not enough pages, nothing changed."""
        before, copies = self.copy(), []
        free = [p for p, r in enumerate(self.refs) if r <= 0][::-1]
        holders, writers = list(self.refs), {}
        for s, r in enumerate(rows):
            if r and self.kv[s] % self.page:
                writers.setdefault(self.used(s)[-1], []).append(s)
        try:
            for s, r in enumerate(rows):
                n = pages_of(self.kv[s], self.page)
                if r and self.kv[s] % self.page:
                    p = self.table[s][n - 1]
                    first = writers[p][0] == s and len(writers[p]) >= holders[p]
                    if holders[p] > 1 and not first:
                        self.table[s][n - 1] = free.pop()
                        self.refs[self.table[s][n - 1]] = 1
                        self.refs[p] -= 1
                        copies.append([p, self.table[s][n - 1]])
                self.kv[s] += r
                for j in range(n, pages_of(self.kv[s], self.page)):
                    self.table[s][j] = free.pop()
                    self.refs[self.table[s][j]] = 1
        except IndexError:
            self.refs, self.kv, self.table = before.refs, before.kv, before.table
            return None
        return copies, len(free)

    def compact(self):
        """(moves, pages held)."""
        held = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(held)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        moves = list(zip(held[n - len(holes):], holes))
        to = dict(moves)
        refs = [0] * len(self.refs)
        for p in held:
            refs[to.get(p, p)] = self.refs[p]
        for s in range(len(self.kv)):
            row = [to.get(p, p) for p in self.used(s)]
            self.table[s][:len(row)] = row
        self.refs = refs
        return [list(m) for m in moves], n


def random_pool(num_pages, page, num_seqs, width, seed):
    """A pool in use: sequences of all lengths, some of them one another's copies."""
    rng = random.Random(seed)
    p = Pool(num_pages, page, num_seqs, width)
    order = list(range(num_pages))
    rng.shuffle(order)
    room = (num_pages * 3) // 4
    for s in range(num_seqs):
        if s and rng.random() < 0.4:             # a copy of an earlier one, perhaps shortened
            t = rng.randrange(s)
            p.kv[s] = rng.choice([p.kv[t], rng.randint(0, p.kv[t])])
            n = pages_of(p.kv[s], page)
            p.table[s][:n] = p.table[t][:n]
            for q in p.used(s):
                p.refs[q] += 1
            continue
        most = min((width - 1) * page, max(0, room - (num_pages - len(order))) * page)
        n = min(most, rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, max(1, most // 4)),
                                  rng.randint(0, most)]))
        p.kv[s] = n
        for j in range(pages_of(n, page)):
            p.table[s][j] = order.pop()
            p.refs[p.table[s][j]] = 1
    return p


def values(logits, scores, last=None, end_token=-1):
    """[groups, beams, vocab] float64: every continuation's value, -inf where there is none."""
    G, K = scores.shape
    x = logits.double()
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    x = x.clamp(max=torch.finfo(torch.float32).max).view(G, K, -1)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), torch.zeros_like(top), top)
    s = torch.exp(x - top).sum(-1, keepdim=True)
    v = torch.where(x > -math.inf, x - top - s.log(), torch.full_like(x, -math.inf))
    if last is not None and end_token >= 0:
        done = (last == end_token).view(G, K)
        v[done] = -math.inf
        v[..., end_token] = torch.where(done, torch.zeros_like(v[..., end_token]),
                                        v[..., end_token])
    score = scores.double()
    score = torch.where(torch.isfinite(score), score, torch.full_like(score, -math.inf))
    return torch.where(torch.isinf(score)[..., None], score[..., None], score[..., None] + v)


def values_bound(logits):
    """What a row's normaliser may be off by, in every one of its values alike.  A term
    2^(x log2 e - ref) with an exponent y <= 0: ex2 within 2 ulp (2^-22), y's two roundings
    (|y| 2^y 2 2^-24 ln 2 < 2^-24); chains of 16 terms of a step, 24 steps, 5 and 8 joins, half a
    step each; the logarithm and the value itself, 2^-22.  Rows with a NaN or +inf, or whose
    largest logit is beyond 2^20, are summed by each thread on its own: chains of vocab / 256."""
    vocab = logits.shape[-1]
    x = torch.where(logits.isnan(), torch.full_like(logits, math.inf), logits).amax(-1)
    plain = bool((x.abs() <= 2.0 ** 20).all())
    chain = 53 if plain else vocab / 256 + 13
    return chain * U32 + 2.0 ** -22 + 2.0 ** -24 + 2.0 ** -22 + (0 if plain else 2.0 ** -21)


def check_selection(out, logits, scores, num_out, last=None, end_token=-1):
    """The outputs of beam_select against the 64-bit values: whole as the definition has them
    but for continuations of different beams that are nearer than the bound."""
    got_s, got_p, got_t = (x.cpu() for x in out)
    logits, scores = logits.cpu(), scores.cpu()
    last = None if last is None else last.cpu()
    G, K = scores.shape
    V = logits.shape[-1]
    val = values(logits, scores, last, end_token)
    # a beam's own order is exact: larger logits, then lower tokens
    x = torch.where(logits.isnan(), torch.full_like(logits, -math.inf), logits).view(G, K, V)
    for g in range(G):
        bound = values_bound(logits[g * K:(g + 1) * K])
        found = min(num_out, int((val[g] > -math.inf).sum()))
        parents, tokens = got_p[g].tolist(), got_t[g].tolist()
        assert parents[found:] == tokens[found:] == [-1] * (num_out - found), (g, found)
        assert bool((got_s[g, found:] == -math.inf).all())
        assert all(g * K <= p < (g + 1) * K for p in parents[:found]), (g, parents)
        beam = [p - g * K for p in parents[:found]]
        want = torch.tensor([float(val[g, k, t]) for k, t in zip(beam, tokens)], dtype=torch.float64)
        assert bool((want > -math.inf).all()), (g, beam, tokens)
        tol = bound + U32 * want.abs()
        # (a value below fp32's range, logits of its lowest and largest value in one row, is
        # -inf rounded to fp32, which is off by more than any tolerance)
        near = torch.where(want.float() == -math.inf, got_s[g, :found] == -math.inf,
                           (got_s[g, :found].double() - want).abs() <= tol)
        assert bool(near.all()), (g, got_s[g].tolist(), want.tolist())
        assert bool((want[1:] <= want[:-1] + 2 * bound).all()), (g, want.tolist())
        left = val[g].clone()
        for k in range(K):
            mine = [t for b, t in zip(beam, tokens) if b == k]
            order = torch.sort(-x[g, k].double(), stable=True).indices[:len(mine)].tolist() \
                if not (last is not None and end_token >= 0 and int(last[g, k]) == end_token) \
                else [end_token]
            assert mine == order[:len(mine)], (g, k, mine, order)
            left[k, mine] = -math.inf
        if found:
            assert float(left.max()) <= float(want[-1]) + 2 * bound, (g, float(left.max()))
