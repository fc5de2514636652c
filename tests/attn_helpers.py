"""Plain 64-bit definitions of the rotation, the paged append and the paged
attention, and the error bounds that their kernels' fp32 arithmetic allows.

A rounding to type t is off by at most half a step, eps(t) / 2 relative to the
value: 2^-24 in fp32, 2^-8 in bf16.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8


def turned(x, positions, freq, rot_scale, interleaved, norm_w=None, eps=1e-6):
    """(value, size) in float64: the rotated heads, and per channel the sum of the two
    absolute channels times rot_scale that a rotation's rounding is relative to."""
    x = x.double()
    if norm_w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * norm_w.double()
    R = 2 * freq.numel()
    i = torch.arange(R // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    t = positions.double()[:, None, None] * freq.double().to(x.device)
    c, s = rot_scale * t.cos(), rot_scale * t.sin()
    y, size = x.clone(), x.abs()
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo] = size[..., hi] = (a.abs() + b.abs()) * abs(rot_scale)
    return y, size


def turned_bound(y, size, dtype):
    """sincospif is within 2 ulp (2^-23) and its argument within half a step of a value of
    at most 1 (pi 2^-24 in the angle); three roundings in the rotation; the norm's sum of up
    to 256 squares in 8 + 5 steps, its division, root and products: at most 16 more."""
    tol = 25 * U32 * size
    return tol + UBF * y.abs() if dtype == torch.bfloat16 else tol


def gather(pages, table_row, n):
    """[n, Hkv, D] float64: keys or values 0 .. n - 1 of one sequence."""
    page = pages.shape[2]
    i = torch.arange(n, device=pages.device)
    return pages[table_row[i // page].long(), :, i % page].double()


def attend(q, k, v, rows, scale, window):
    """(out, size, spread) in float64 for one sequence: q [rows, Hq, D], k and v [n, Hkv, D].
    size = sum p |v| / sum p; spread = the largest scale * sum |q||k| of a row."""
    n, Hkv, D = k.shape
    Hq = q.shape[1]
    G = Hq // Hkv
    q = q.double().view(rows, Hkv, G, D)
    s = torch.einsum("rhgd,nhd->hgrn", q, k) * scale
    big = torch.einsum("rhgd,nhd->hgrn", q.abs(), k.abs()) * scale
    i = n - rows + torch.arange(rows, device=k.device)[:, None]
    j = torch.arange(n, device=k.device)[None, :]
    see = (j <= i) & ((j > i - window) if window else torch.ones_like(j, dtype=torch.bool))
    s = s.masked_fill(~see, -math.inf)
    m = s.amax(-1, keepdim=True) if n else torch.full((Hkv, G, rows, 1), -math.inf).to(s)
    p = torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / l, torch.zeros_like(p))
    out = torch.einsum("hgrn,nhd->rhgd", p, v).reshape(rows, Hq, D)
    size = torch.einsum("hgrn,nhd->rhgd", p, v.abs()).reshape(rows, Hq, D)
    spread = big.masked_fill(~see, 0).amax(-1) if n else torch.zeros(Hkv, G, rows).to(s)
    return out, size, spread.permute(2, 0, 1).reshape(rows, Hq, 1)


def attend_bound(out, size, spread, n, D, out_dtype, p_bf16):
    """Scores: D fp32 additions of products, each within 2^-23 (a tensor core may truncate):
    p is off by twice that (in p and in the sum); ex2 within 2 ulp and its argument's
    rounding (of exponents below 2^8: 2^-16); the sums of n products and of n terms, in runs
    of at most n / 16 + 64 additions; p in bf16 (2^-8) or in two bf16 halves (2^-16)."""
    rel = 2 * (D + 8) * 2 * U32 * spread + 2.0 ** -15 + 2 * (n / 16 + 64) * 2 * U32
    tol = size * (rel + (UBF if p_bf16 else 2.0 ** -16))
    return tol + UBF * out.abs() if out_dtype == torch.bfloat16 else tol


class Paged:
    """A ragged batch over a shuffled page pool whose unused slots hold NaN."""

    def __init__(self, rows, kv, Hq, Hkv, D, page, dev, seed=0, joined=False, spare=2):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.rows, self.kv, self.Hq, self.Hkv, self.D, self.page = rows, kv, Hq, Hkv, D, page
        need = [-(-n // page) for n in kv]
        self.pool = sum(need) + spare
        ids = torch.randperm(self.pool, generator=g).to(torch.int32)
        width = max(need + [1]) + 1
        # entries past a sequence's pages name no page at all
        self.page_table = torch.full((len(rows), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.page_table[b, :n] = ids[at:at + n]
            at += n
        start = [0]
        for n in rows:
            start.append(start[-1] + n)
        self.T = start[-1]
        self.row_start = torch.tensor(start, dtype=torch.int32, device=dev)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=dev)
        self.max_rows = max(rows + [1])
        shape = (self.pool, Hkv, page, D)
        if joined:  # keys and values of a page side by side in one buffer
            buf = torch.full((self.pool, 2) + shape[1:], math.nan, dtype=torch.bfloat16, device=dev)
            self.k_pages, self.v_pages = buf[:, 0], buf[:, 1]
        else:
            self.k_pages = torch.full(shape, math.nan, dtype=torch.bfloat16, device=dev)
            self.v_pages = torch.full(shape, math.nan, dtype=torch.bfloat16, device=dev)
        gd = torch.Generator(device=dev)
        gd.manual_seed(seed + 1)
        for b, n in enumerate(kv):
            if n == 0:
                continue
            i = torch.arange(n, device=dev)
            pg = self.page_table.to(dev)[b, i // page].long()
            for pages, gain in ((self.k_pages, 1.5), (self.v_pages, 1.0)):
                pages[pg, :, i % page] = (torch.randn(n, Hkv, D, generator=gd, device=dev) *
                                          gain).to(torch.bfloat16)
        self.q = torch.randn(self.T, Hq, D, generator=gd, device=dev).to(torch.bfloat16)
        self.page_table = self.page_table.to(dev)

    def check(self, out, p_bf16, window=0, scale=None, q=None):
        """Every row of `out` against the 64-bit definition, within its bound."""
        scale = self.D ** -0.5 if scale is None else scale
        q = self.q if q is None else q
        at, worst = 0, 0.0
        for b, (r, n) in enumerate(zip(self.rows, self.kv)):
            if r == 0:
                continue
            k = gather(self.k_pages, self.page_table[b], n)
            v = gather(self.v_pages, self.page_table[b], n)
            ref, size, spread = attend(q[at:at + r], k, v, r, scale, window)
            tol = attend_bound(ref, size, spread, n, self.D, out.dtype, p_bf16)
            err = (out[at:at + r].double() - ref).abs()
            bad = ~(err <= tol)
            assert not bad.any(), (f"sequence {b} (rows {r}, keys {n}): {int(bad.sum())} values "
                                   f"off, first at {bad.nonzero()[0].tolist()}, "
                                   f"worst {float((err - tol).max()):.3e} over its bound")
            worst = max(worst, float((err / tol.clamp_min(1e-30)).max()))
            at += r
        return worst
