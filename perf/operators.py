"""The attention operators beside the expert layer, measured.

A decoder layer that uses this library's expert layer needs three more steps
between its projections: the position rotation of the heads, the write of new
keys and values into the paged cache (with the rotation on the way), and the
attention of the new rows over that cache.  This file holds their cases, their
plain form in elementary torch operations, and their definition in 64 bits.

Shapes: x [T, H, D]; pages [P, Hkv, page, D]; sequence b owns the rows
row_start[b] .. row_start[b + 1] - 1 of q, k and v, its length with these rows
is kv_len[b], and key i of it lies in page page_table[b, i // page] at slot
i % page.  A row sees the keys up to its own, the last `window` of them where
window is not 0.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
EPS = 1e-6
WORKSPACE = 64 << 20      # bytes of the attention's workspace, zeroed once


# --------------------------------------------------------------- the cases

def listed():
    return [
        # one decoded token's query heads: what counts is the call's latency
        dict(name="rope_token", op="rope", T=1, H=64, D=128, R=128, pairs="half", fp32=False,
             norm=True, far=40_000, stretch=1.0, seed=1),
        # the heads of a long prompt, a quarter of each rotated, positions far
        # past the trained length (frequencies stretched by parts)
        dict(name="rope_prompt", op="rope", T=16_411, H=40, D=128, R=32, pairs="adjacent",
             fp32=False, norm=False, far=1_000_000, stretch=16.0, seed=2),
        # a middle-sized batch of fp32 heads with their norm
        dict(name="rope_fp32", op="rope", T=2_501, H=36, D=64, R=64, pairs="half", fp32=True,
             norm=True, far=131_072, stretch=1.0, seed=3),
        # one step of a decode batch: one new row for each of 128 sequences
        dict(name="append_step", op="append", B=128, rows="one", longest=4_000, Hq=64, Hkv=4,
             D=128, R=128, page=16, pairs="half", fp32=False, norm=True, seed=4),
        # the chunks of several prompts, ragged, fp32 projections
        dict(name="append_chunks", op="append", B=6, rows="ragged", longest=6_001, Hq=32, Hkv=8,
             D=128, R=128, page=64, pairs="half", fp32=True, norm=False, seed=5),
        # the next token of one short conversation
        dict(name="attend_token", op="attend", B=1, rows="one", longest=777, Hq=64, Hkv=4, D=128,
             page=16, window=0, seed=6),
        # a full decode batch of conversations of all lengths
        dict(name="attend_batch", op="attend", B=96, rows="one", longest=16_001, Hq=64, Hkv=4,
             D=128, page=64, window=0, seed=7),
        # the next token after one very long document
        dict(name="attend_long", op="attend", B=1, rows="one", longest=500_003, Hq=32, Hkv=8,
             D=128, page=128, window=0, seed=8),
        # several drafted tokens of each sequence checked at once
        dict(name="attend_drafts", op="attend", B=24, rows="five", longest=9_999, Hq=32, Hkv=8,
             D=128, page=32, window=0, seed=9),
        # a prompt's chunk that shares its step with the next tokens of others
        dict(name="attend_mixed", op="attend", B=33, rows="mixed", longest=8_000, Hq=64, Hkv=4,
             D=128, page=64, window=0, seed=10),
        # the chunks of two long prompts
        dict(name="attend_prompt", op="attend", B=2, rows="ragged", longest=9_001, Hq=64, Hkv=4,
             D=128, page=64, window=0, seed=15),
        # prompts under a sliding window, small heads, small pages
        dict(name="attend_window", op="attend", B=5, rows="ragged", longest=5_003, Hq=40, Hkv=8,
             D=64, page=16, window=1_024, seed=12),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    seed = rng.randrange(1 << 30)
    if op == "rope":
        D = rng.choice([64, 128])
        return dict(op=op, T=_spread(rng, 1, 16_000), H=rng.randint(1, 40), D=D,
                    R=rng.choice([D, D // 2, D // 4, 24]), pairs=rng.choice(["half", "adjacent"]),
                    fp32=rng.random() < 0.3, norm=rng.random() < 0.5,
                    far=_spread(rng, 100, 1_000_000), stretch=rng.choice([1.0, 4.0, 16.0]),
                    seed=seed)
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    D = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        rows = rng.choice(["one", "ragged"])
        return dict(op=op, B=_spread(rng, 1, 200) if rows == "one" else rng.randint(1, 6),
                    rows=rows, longest=_spread(rng, 100, 6_000), Hq=Hkv * G, Hkv=Hkv, D=D,
                    R=rng.choice([D, D // 2]), page=page, pairs=rng.choice(["half", "adjacent"]),
                    fp32=rng.random() < 0.3, norm=rng.random() < 0.5, seed=seed)
    rows = rng.choice(["one", "one", "five", "mixed", "ragged"])
    B = {"one": _spread(rng, 1, 128), "five": rng.randint(1, 32), "mixed": rng.randint(2, 33),
         "ragged": rng.randint(1, 2)}[rows]
    longest = _spread(rng, 50, 9_000 if rows != "one" else 16_000)
    return dict(op=op, B=B, rows=rows, longest=longest, Hq=Hkv * min(G, 64 // Hkv), Hkv=Hkv, D=D,
                page=page, window=rng.choice([0, 0, 0, 1_000]), seed=seed)


def lengths(case):
    """(rows, kv_len) of every sequence, as lists: they are the case's own."""
    rng = random.Random(case["seed"])
    B, longest, kind = case["B"], case["longest"], case["rows"]
    kv = [longest if b == 0 else _spread(rng, 1, longest) for b in range(B)]
    if kind == "one":
        rows = [1] * B
    elif kind == "five":
        rows = [5] * B
        kv = [max(n, 5) for n in kv]
    elif kind == "mixed":      # one long chunk, one idle sequence, single rows
        rows = [1] * B
        rows[0] = max(1, longest // 4)
        rows[-1] = 0
        order = list(range(B))
        rng.shuffle(order)
        rows, kv = [rows[i] for i in order], [kv[i] for i in order]
    else:                      # chunks: a whole prompt first, then parts of others
        rows = [n if b == 0 else max(1, int(n * rng.uniform(0.3, 1.0))) for b, n in enumerate(kv)]
    return rows, kv


# --------------------------------------------------------------- the inputs

def frequencies(R, theta, stretch):
    """Radians a position turns each of the R / 2 pairs: theta^(-2i/R); with a
    stretch s > 1 the slow pairs are slowed by s, the fast ones kept, and those
    between blended by a ramp over the turns they make in 4096 positions (from
    32 down to 1).  Also the factor on cosine and sine, 0.1 ln s + 1."""
    i = torch.arange(R // 2, dtype=torch.float64)
    f = theta ** (-2.0 * i / R)
    if stretch == 1.0:
        return f, 1.0
    at = [R * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32, 1)]
    low, high = max(0, math.floor(at[0])), min(R - 1, math.ceil(at[1]))
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f / stretch * ramp + f * (1 - ramp), 0.1 * math.log(stretch) + 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def heads(T, H, D):
        # heads as projections give them: most channels alike, a few of each
        # head much larger and with a mean of their own
        mean = randn(1, H, D) * (torch.rand(1, H, D, generator=g, device=DEV) < 0.06) * 3
        return randn(T, H, D) + mean

    s = dict(case)
    if case["op"] in ("rope", "append"):
        dtype = torch.float32 if case["fp32"] else torch.bfloat16
        freq, factor = frequencies(case["R"], 1e6, case.get("stretch", 1.0))
        # the rotation's table: each frequency in 2^-64 turns a position
        s.update(freq=freq.to(DEV), factor=factor,
                 table=(freq / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEV))
        s["norm_q"] = s["norm_k"] = None
        if case["norm"]:
            s["norm_q"] = (1 + 0.2 * randn(case["D"])).to(torch.bfloat16)
            s["norm_k"] = (1 + 0.2 * randn(case["D"])).to(torch.bfloat16)
    if case["op"] == "rope":
        T = case["T"]
        s["x"] = heads(T, case["H"], case["D"]).to(dtype)
        at = torch.randint(0, case["far"], (1,), generator=g, device=DEV)
        s["positions"] = ((at + torch.arange(T, device=DEV)) % case["far"]).to(torch.int32)
        return s
    rows, kv = lengths(case)
    B, Hq, Hkv, D, page = case["B"], case["Hq"], case["Hkv"], case["D"], case["page"]
    T = sum(rows)
    need = [-(-n // page) for n in kv]
    pool = sum(need) + 3
    ids = torch.randperm(pool, generator=g, device=DEV).to(torch.int32).cpu()
    page_table = torch.zeros(B, max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        page_table[b, :n] = ids[at:at + n]
        at += n
    start = [0]
    for n in rows:
        start.append(start[-1] + n)
    s.update(rows=rows, kv=kv, max_rows=max(rows), page_table=page_table.to(DEV),
             row_start=torch.tensor(start, dtype=torch.int32, device=DEV),
             kv_len=torch.tensor(kv, dtype=torch.int32, device=DEV))
    mean = randn(1, Hkv, 1, D) * (torch.rand(1, Hkv, 1, D, generator=g, device=DEV) < 0.06) * 3
    s["k_pages"] = (randn(pool, Hkv, page, D) + mean).to(torch.bfloat16)
    s["v_pages"] = randn(pool, Hkv, page, D).to(torch.bfloat16)
    if case["op"] == "append":
        # one projection's output, split: q, k and v are strided views of it
        qkv = heads(T, Hq + 2 * Hkv, D).to(dtype)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s["q"] = heads(T, Hq, D).to(torch.bfloat16)
        s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------- the plain form

def plain_rotate(x, positions, s, weight):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    R = 2 * s["freq"].numel()
    angle = positions.double()[:, None] * s["freq"]
    cos = (angle.cos() * s["factor"]).float()[:, None]
    sin = (angle.sin() * s["factor"]).float()[:, None]
    if s["pairs"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., R:]], -1)


def plain_rope(s):
    return plain_rotate(s["x"], s["positions"], s, s["norm_q"]).to(s["x"].dtype)


def plain_append(s):
    T, page = s["q"].shape[0], s["page"]
    row = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["row_start"].long(), row, right=True) - 1
    index = s["kv_len"][b] - s["row_start"][b + 1] + row      # key index of each row
    q = plain_rotate(s["q"], index, s, s["norm_q"]).to(torch.bfloat16)
    k = plain_rotate(s["k"], index, s, s["norm_k"]).to(torch.bfloat16)
    at = s["page_table"][b, index // page].long()
    s["k_pages"][at, :, index % page] = k
    s["v_pages"][at, :, index % page] = s["v"].to(torch.bfloat16)
    return q, s["k_pages"], s["v_pages"]


def plain_keys(pages, table):
    """[n, L, Hkv, D] in 32 bits: the pages of `table` [n, p] in order."""
    x = pages[table.long()].float()                           # [n, p, Hkv, page, D]
    return x.transpose(2, 3).flatten(1, 2)


def plain_attend_equal(q, k, v, kv_len, window):
    """q [n, r, Hq, D], the last r rows of n sequences; k, v [n, L, Hkv, D]."""
    n, r, Hq, D = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    q = q.float().reshape(n, r, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(D)        # [n, Hkv, G r, L]
    score = score.view(n, Hkv, Hq // Hkv, r, L)
    key = torch.arange(L, device=DEV)
    last = (kv_len[:, None] - r + torch.arange(r, device=DEV))[..., None]   # [n, r, 1]
    seen = key <= last
    if window:
        seen = seen & (key > last - window)
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top.isinf(), 0.0, top)).exp()
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill((key >= kv_len[:, None])[..., None, None], 0.0)
    out = (p.flatten(2, 3) @ v.transpose(1, 2)).view(n, Hkv, Hq // Hkv, r, D)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(n, r, Hq, D)


def plain_attend(s):
    q, rows, kv, page = s["q"], s["rows"], s["kv"], s["page"]
    if min(rows) == max(rows):                                # one batched product
        out = plain_attend_equal(q.view(len(rows), rows[0], *q.shape[1:]),
                                 plain_keys(s["k_pages"], s["page_table"]),
                                 plain_keys(s["v_pages"], s["page_table"]), s["kv_len"],
                                 s["window"])
        return out.reshape(q.shape).to(torch.bfloat16)
    out, at = torch.empty_like(q), 0
    for b, r in enumerate(rows):
        if r:
            table = s["page_table"][b:b + 1, :-(-kv[b] // page)]
            out[at:at + r] = plain_attend_equal(q[None, at:at + r],
                                                plain_keys(s["k_pages"], table),
                                                plain_keys(s["v_pages"], table),
                                                s["kv_len"][b:b + 1], s["window"])[0]
        at += r
    return out


def run(s):
    op = s["op"]
    if not own:
        return {"rope": plain_rope, "append": plain_append, "attend": plain_attend}[op](s)
    import bit_expert_weight_gb300.smoe as S
    if op == "rope":
        return S.rope(s["x"], s["positions"], s["table"], rot_scale=s["factor"],
                      interleaved=s["pairs"] == "adjacent", norm_w=s["norm_q"], eps=EPS)
    if op == "append":
        q = S.kv_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["row_start"],
                        s["kv_len"], s["page_table"], table=s["table"], rot_scale=s["factor"],
                        interleaved=s["pairs"] == "adjacent", q_norm=s["norm_q"],
                        k_norm=s["norm_k"], eps=EPS)
        return q, s["k_pages"], s["v_pages"]
    return S.attention(s["q"], s["k_pages"], s["v_pages"], s["row_start"], s["kv_len"],
                       s["page_table"], s["max_rows"], s["workspace"], window=s["window"])


# --------------------------------------------------------------- work and definition

def work(case):
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["D"]
        return {"bytes": 2 * n * (4 if case["fp32"] else 2) + 4 * case["T"], "flops": 6 * n}
    rows, kv = lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        n = sum(rows) * (Hq + 2 * Hkv) * D
        return {"bytes": n * (6 if case["fp32"] else 4), "flops": 6 * n}
    window, keys, pairs = case["window"], 0, 0
    for r, n in zip(rows, kv):
        first = n - r + 1                                     # keys that the first row sees
        if r and window:
            keys += min(n, window + r - 1)
            under = max(0, min(n, window) - first + 1)        # rows that see fewer than window + 1
            pairs += under * (first + first + under - 1) // 2 + (r - under) * window
        elif r:
            keys += n
            pairs += r * (first + n) // 2
    return {"bytes": 2 * 2 * keys * Hkv * D + 2 * 2 * sum(rows) * Hq * D,
            "flops": 4 * pairs * Hq * D}


def exact_turned(x, positions, s, weight):
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    R = 2 * s["freq"].numel()
    pair = torch.arange(R // 2, device=DEV)
    lo, hi = (pair, pair + R // 2) if s["pairs"] == "half" else (2 * pair, 2 * pair + 1)
    turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=DEV),
                       positions.double()[:, None, None] * s["freq"])
    z = torch.complex(x[..., lo], x[..., hi]) * turn
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return exact_turned(s["x"], s["positions"], s, s["norm_q"])
    rows, kv, page, table = s["rows"], s["kv"], s["page"], s["page_table"].long()
    if case["op"] == "append":
        index = torch.cat([torch.arange(n - r, n, device=DEV) for r, n in zip(rows, kv)])
        owner = torch.cat([torch.full((r,), b, device=DEV) for b, r in enumerate(rows)])
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        slot = (table[owner, torch.div(index, page, rounding_mode="floor")], index % page)
        k_pages.transpose(1, 2)[slot] = exact_turned(s["k"], index, s, s["norm_k"])
        v_pages.transpose(1, 2)[slot] = s["v"].double()
        return exact_turned(s["q"], index, s, s["norm_q"]), k_pages, v_pages
    Hkv, G, D, at = case["Hkv"], case["Hq"] // case["Hkv"], case["D"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (r, n) in enumerate(zip(rows, kv)):
        key = torch.arange(n, device=DEV)
        slot = (table[b, key // page], key % page)
        own_key = torch.arange(n - r, n, device=DEV)
        back = own_key[:, None] - key                         # how far back a key lies
        unseen = (back < 0) | (back >= (case["window"] or n))
        for h in range(Hkv if r else 0):
            k, v = (x[slot[0], h, slot[1]].double() for x in (s["k_pages"], s["v_pages"]))
            for j in range(h * G, (h + 1) * G):
                log = s["q"][at:at + r, j].double() @ (k.T / math.sqrt(D))
                log[unseen] = -math.inf
                log -= log.logsumexp(-1, keepdim=True)
                out[at:at + r, j] = log.exp() @ v
        at += r
    return out
