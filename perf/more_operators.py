"""Beam search over the paged cache and the upkeep of its pages, measured.

Next to the attention over a paged cache, a serving program needs: the choice of
the next tokens over beams and vocabulary, the sequences' pages reordered after
it and shared where beams came from the same one, room for the next rows, pages
copied where a shared one is about to be written, and the pool compacted now and
then.  This file holds their cases, their plain form in elementary torch
operations, and their definition.

Shapes: logits [G K, V] (K beams of G groups); refs [P], how many sequences hold
a page; kv_len [S]; page_table [S, W], of which sequence s uses the first
ceil(kv_len[s] / page) entries; pages [P, Hkv, page, D].
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
END = 2                   # the token that ends a sequence
WORKSPACE = 32 << 20      # bytes of the selection's workspace, zeroed once


# --------------------------------------------------------------- the cases

def listed():
    return [
        # the next tokens of one request's four beams: what counts is latency
        dict(name="select_one", op="select", G=1, K=4, V=32_000, N=4, fp32=False, allowed=1.0,
             seed=1),
        # a full batch of requests, as many candidates as the beams need when all of them end
        dict(name="select_batch", op="select", G=64, K=8, V=151_936, N=16, fp32=False, allowed=1.0,
             seed=2),
        # an odd vocabulary, so that rows start anywhere, in fp32
        dict(name="select_odd", op="select", G=12, K=5, V=100_003, N=10, fp32=True, allowed=1.0,
             seed=3),
        # constrained decoding: most tokens are masked with the type's lowest value
        dict(name="select_masked", op="select", G=20, K=16, V=65_536, N=32, fp32=False,
             allowed=0.003, seed=4),
        # one request's beams reordered
        dict(name="fork_group", op="fork", G=1, K=4, longest=2_000, page=16, spare=300, seed=5),
        # a full batch of long requests reordered, some of them finished and let go
        dict(name="fork_batch", op="fork", G=64, K=8, longest=16_001, page=16, spare=5_000, seed=6),
        # a step of a batch's beams: cut back, reordered, one more row each
        dict(name="reserve_step", op="reserve", G=48, K=5, longest=9_999, page=16, spare=90_000,
             rows="one", seed=7),
        # chunks of prompts beside the next tokens of others, in a large pool
        dict(name="reserve_chunks", op="reserve", G=200, K=1, longest=20_011, page=16,
             spare=400_000, rows="chunks", seed=8),
        # the pages that a step's beams write apart, in a few layers at once
        dict(name="copy_step", op="copy", L=4, n=12, most=64, pool=200, Hkv=4, D=128, page=16,
             joined=True, seed=9),
        # a part of a pool moved, in two layers
        dict(name="copy_pool", op="copy", L=2, n=601, most=700, pool=1_300, Hkv=8, D=128, page=64,
             joined=False, seed=10),
        # a small pool closed up
        dict(name="compact_small", op="compact", G=30, K=1, longest=1_500, page=16, spare=700,
             seed=11),
        # a large one, whose pages are partly shared
        dict(name="compact_large", op="compact", G=120, K=4, longest=20_000, page=16,
             spare=300_000, seed=12),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["select", "select", "select", "fork", "reserve", "copy", "compact"])
    seed = rng.randrange(1 << 30)
    if op == "select":
        V = _spread(rng, 1_000, 151_936)
        K = rng.choice([1, 2, 3, 4, 5, 8, 16])
        fp32 = rng.random() < 0.4
        G = _spread(rng, 1, max(1, min(64, 70_000_000 // (K * V * (2 if fp32 else 1)))))
        return dict(op=op, G=G, K=K, V=V, N=rng.choice([K, 2 * K, K + 1]), fp32=fp32,
                    allowed=rng.choice([1.0, 1.0, 0.01]), seed=seed)
    page = rng.choice([16, 32, 64, 128])
    if op == "copy":
        n = _spread(rng, 1, 400)
        return dict(op=op, L=rng.randint(1, 3), n=n, most=n + rng.choice([0, 1, 50]),
                    pool=2 * n + rng.randint(0, 100), Hkv=rng.choice([1, 2, 4, 8]),
                    D=rng.choice([64, 128]), page=min(page, 64), joined=rng.random() < 0.5,
                    seed=seed)
    case = dict(op=op, G=_spread(rng, 1, 64), K=rng.choice([2, 3, 4, 5, 8]),
                longest=_spread(rng, 40, 16_000), page=page, spare=_spread(rng, 10, 100_000),
                seed=seed)
    if op == "reserve":
        rows = rng.choice(["one", "chunks"])
        case.update(rows=rows, spare=case["spare"] + 40_000)
        if rows == "chunks":
            case["K"] = 1
    return case


def pages_of(keys, page):
    return -(-keys // page)


def sequences(case):
    """The case's own sizes: (keys of every sequence, how many of its pages it shares with its
    group, parents, rows to come)."""
    rng = random.Random(case["seed"])
    G, K, page = case["G"], case["K"], case["page"]
    kv, shared, parent, rows = [], [], [], []
    for g in range(G):
        n = case["longest"] if g == 0 else _spread(rng, 1, case["longest"])
        common = int(0.75 * n) // page if K > 1 else 0       # the prompt's full pages
        gone = case["op"] == "fork" and g > 0 and rng.random() < 1 / 16
        stay = rng.randint(1, K)                             # beams that go on; the others
        for k in range(K):                                   # become copies of one of them
            kv.append(n)
            shared.append(common)
            at = k if k < stay else rng.randrange(stay)
            parent.append(-1 if gone else g * K + at)
            if case.get("rows") == "chunks":
                rows.append(rng.choice([0, 1, 1, _spread(rng, 1, case["longest"] // 4 + 1)]))
            else:
                rows.append(1)
    return kv, shared, parent, rows


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    i32 = torch.int32

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    s = dict(case)
    if case["op"] == "select":
        G, K, V, N = case["G"], case["K"], case["V"], case["N"]
        dtype = torch.float32 if case["fp32"] else torch.bfloat16
        # logits as a head gives them: a bulk, and a few tokens that stand out in each row
        x = 2.0 * randn(G * K, V)
        x += (rand(G * K, V) < 20 / V) * 6.0 * rand(G * K, V)
        if case["allowed"] < 1:
            x[rand(G * K, V) >= case["allowed"]] = torch.finfo(dtype).min
        x[:, 0] = -math.inf                                  # never said
        s["logits"] = x.to(dtype)
        s["scores"] = -20 - 3 * rand(G, K)
        s["last"] = torch.randint(3, V, (G, K), generator=g, device=DEV, dtype=i32)
        s["last"][rand(G, K) < 0.1] = END                    # finished beams
        dead = rand(G, K) < 0.05                             # beams that lead nowhere
        dead[:, 0] = False
        s["scores"][dead] = -math.inf
        s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV)
        s["out"] = (torch.zeros(G, N, device=DEV), torch.zeros(G, N, dtype=i32, device=DEV),
                    torch.zeros(G, N, dtype=i32, device=DEV))
        return s
    if case["op"] == "copy":
        P, Hkv, page, D = case["pool"], case["Hkv"], case["page"], case["D"]
        s["k_pages"], s["v_pages"] = [], []
        for _ in range(case["L"]):
            if case["joined"]:                               # keys and values of a page together
                both = randn(P, 2, Hkv, page, D).to(torch.bfloat16)
                s["k_pages"].append(both[:, 0])
                s["v_pages"].append(both[:, 1])
            else:
                s["k_pages"].append(randn(P, Hkv, page, D).to(torch.bfloat16))
                s["v_pages"].append(randn(P, Hkv, page, D).to(torch.bfloat16))
        ids = torch.randperm(P, generator=g, device=DEV)[:2 * case["n"]].to(i32)
        s["copies"] = torch.full((case["most"], 2), -1, dtype=i32, device=DEV)
        s["copies"][:case["n"]] = ids.view(-1, 2)
        s["counts"] = torch.tensor([case["n"], 0], dtype=i32, device=DEV)
        return s
    kv, shared, parent, rows = sequences(case)
    page, K, S = case["page"], case["K"], case["G"] * case["K"]
    need = [pages_of(n, page) for n in kv]
    used = sum(n - c for n, c in zip(need, shared)) + sum(shared[::K])
    more = [pages_of(n + r, page) for n, r in zip(kv, rows)]
    pool = used + case["spare"] + sum(more) - sum(need)
    ids = torch.randperm(pool, generator=g, device=DEV).to(i32).cpu()
    table = torch.full((S, max(more) + 1), -1, dtype=i32)
    at = 0
    for b, (n, c) in enumerate(zip(need, shared)):
        if b % K == 0:
            table[b:b + K, :c] = ids[at:at + c]
            at += c
        table[b, c:n] = ids[at:at + n - c]
        at += n - c
    held = table[torch.arange(table.shape[1]) < torch.tensor(need)[:, None]]
    start = [0]
    for r in rows:
        start.append(start[-1] + r)
    s.update(kv_len=torch.tensor(kv, dtype=i32, device=DEV), page_table=table.to(DEV),
             refs=torch.bincount(held.long(), minlength=pool).to(i32).to(DEV),
             counts=torch.zeros(2, dtype=i32, device=DEV))
    if case["op"] == "compact":
        s.update(refs_out=s["refs"].clone(), table_out=s["page_table"].clone(),
                 copies=torch.zeros(pool // 2, 2, dtype=i32, device=DEV))
    else:
        s.update(parent=torch.tensor(parent, dtype=i32, device=DEV))
    if case["op"] == "reserve":
        # every step begins with what earlier ones left: the rows that it adds are cut off
        # again by the next one, as those of refused drafts are
        s.update(keep=s["kv_len"].clone(), copies=torch.zeros(S, 2, dtype=i32, device=DEV),
                 row_start=torch.tensor(start, dtype=i32, device=DEV))
    return s


# --------------------------------------------------------------- the plain form

def plain_select(s):
    G, K, V, N = s["G"], s["K"], s["V"], s["N"]
    # in 64 bits: candidates of several beams may lie close to one another
    x, none = s["logits"].double(), -math.inf
    top = x.amax(-1, keepdim=True)
    x = x - torch.where(top.isinf(), 0.0, top)
    x = x - x.exp().sum(-1, keepdim=True).log()
    finished = (s["last"] == END).view(-1, 1)
    x = torch.where(finished, torch.where(torch.arange(V, device=DEV) == END, 0.0, none), x)
    score = s["scores"].double().view(-1, 1)
    value = torch.where(score == none, none, score + x).view(G, K * V)
    value, at = value.sort(dim=-1, descending=True, stable=True)
    value, at = value[:, :N], at[:, :N]
    beam = at // V + K * torch.arange(G, device=DEV)[:, None]
    found = value > none
    return (value.float(), torch.where(found, beam, -1).to(torch.int32),
            torch.where(found, at % V, -1).to(torch.int32))


def plain_count(refs, table, used, by):
    """Adds `by` (of table's shape or 1) to the holders of the table's used entries."""
    refs.scatter_add_(0, table.clamp_min(0).long().flatten(),
                      torch.where(used, by, 0).to(torch.int32).flatten())


def plain_fork(s, keep=None):
    table, kv, refs, page = s["page_table"], s["kv_len"], s["refs"], s["page"]
    parent = s["parent"].long()
    column = torch.arange(table.shape[1], device=DEV)
    there, source = parent >= 0, parent.clamp_min(0)
    length = torch.where(there, kv[source], 0)
    if keep is not None:
        length = torch.minimum(length, keep.clamp_min(0))
    new = column < ((length + page - 1) // page)[:, None]
    plain_count(refs, table, column < ((kv + page - 1) // page)[:, None], -1)
    table.copy_(torch.where(new, table[source], table))
    plain_count(refs, table, new, 1)
    kv.copy_(length)
    return kv, table, refs


def plain_reserve(s):
    table, kv, refs, page = s["page_table"], s["kv_len"], s["refs"], s["page"]
    S, W = table.shape
    rows = s["row_start"].diff()
    had, will = (kv + page - 1) // page, (kv + rows + page - 1) // page
    last = table.gather(1, (had - 1).clamp_min(0).long()[:, None])[:, 0].clamp_min(0).long()
    writes = (rows > 0) & (kv % page > 0)
    same = (last[:, None] == last) & writes[:, None] & writes
    first = ~torch.tril(same, -1).any(1)                      # none before it writes there too
    apart = writes & ~((refs[last] == same.sum(1)) & first) & (refs[last] > 1)
    need = will - had + apart.int()
    base = need.cumsum(0) - need
    free = refs == 0
    ids = torch.argsort(free.int(), descending=True, stable=True).to(torch.int32)
    column = torch.arange(W, device=DEV)
    from_ = had - apart.int()
    fresh = (column >= from_[:, None]) & (column < will[:, None])
    rank = (base[:, None] + column - from_[:, None]).clamp(0, ids.numel() - 1)
    table.copy_(torch.where(fresh, ids[rank.long()], table))
    plain_count(refs, last, apart, -1)
    plain_count(refs, table, fresh, 1)
    kv += rows
    # the copies, in order of their sequences
    order = torch.argsort(apart.int(), descending=True, stable=True)
    pairs = torch.stack([last.to(torch.int32), ids[base.clamp_max(ids.numel() - 1).long()]], -1)
    n = apart.sum()
    s["copies"].copy_(torch.where((torch.arange(S, device=DEV) < n)[:, None], pairs[order],
                                  s["copies"]))
    s["counts"].copy_(torch.stack([n, free.sum() - need.sum()]))
    return kv, table, refs, s["copies"], s["counts"]


def plain_copy(s):
    valid = torch.arange(s["most"], device=DEV) < s["counts"][0]
    pairs = torch.where(valid[:, None], s["copies"], s["copies"][:1]).long()
    for pages in s["k_pages"] + s["v_pages"]:
        pages[pairs[:, 1]] = pages[pairs[:, 0]]
    return s["k_pages"], s["v_pages"]


def plain_compact(s):
    table, kv, refs, page = s["page_table"], s["kv_len"], s["refs"], s["page"]
    P, most = refs.numel(), s["copies"].shape[0]
    page_id = torch.arange(P, device=DEV)
    held = refs > 0
    n = held.sum()
    to = torch.argsort((~held & (page_id < n)).int(), descending=True, stable=True)
    move = held & (page_id >= n)
    source = torch.argsort(move.int(), descending=True, stable=True)
    count = move.sum()
    new_id = torch.where(move, to[(move.cumsum(0) - 1).clamp_min(0)], page_id)
    s["refs_out"].zero_().scatter_add_(0, new_id, refs)
    used = torch.arange(table.shape[1], device=DEV) < ((kv + page - 1) // page)[:, None]
    s["table_out"].copy_(torch.where(used, new_id[table.clamp_min(0).long()], s["table_out"]))
    pairs = torch.stack([source, to], -1)[:most].to(torch.int32)
    s["copies"].copy_(torch.where((torch.arange(most, device=DEV) < count)[:, None], pairs,
                                  s["copies"]))
    s["counts"].copy_(torch.stack([count, n]))
    return s["refs_out"], s["table_out"], s["copies"], s["counts"]


def run(s):
    op = s["op"]
    if not own:
        if op == "reserve":
            plain_fork(s, s["keep"])
            return plain_reserve(s)
        return {"select": plain_select, "fork": plain_fork, "copy": plain_copy,
                "compact": plain_compact}[op](s)
    import bit_expert_weight_gb300.smoe as S
    if op == "select":
        return S.beam_select(s["logits"], s["scores"], s["N"], s["workspace"], last=s["last"],
                             end_token=END, out=s["out"])
    if op == "copy":
        S.pages_copy(s["k_pages"], s["v_pages"], s["copies"], s["counts"])
        return s["k_pages"], s["v_pages"]
    pool = (s["refs"], s["kv_len"], s["page_table"], s["page"])
    if op == "compact":
        S.pages_compact(*pool, s["copies"], s["counts"], refs_out=s["refs_out"],
                        page_table_out=s["table_out"])
        return s["refs_out"], s["table_out"], s["copies"], s["counts"]
    S.pages_fork(*pool, s["parent"], keep=s.get("keep"))
    if op == "fork":
        return s["kv_len"], s["page_table"], s["refs"]
    S.pages_reserve(*pool, s["row_start"], s["copies"], s["counts"])
    return s["kv_len"], s["page_table"], s["refs"], s["copies"], s["counts"]


# --------------------------------------------------------------- work and definition

def work(case):
    if case["op"] == "select":
        n = case["G"] * case["K"] * case["V"]
        return {"bytes": n * (4 if case["fp32"] else 2) + 12 * case["G"] * case["N"],
                "flops": 4 * n}
    if case["op"] == "copy":
        n = case["L"] * case["n"] * 2 * case["Hkv"] * case["page"] * case["D"] * 2
        return {"bytes": 2 * n, "flops": 0}
    kv, shared, parent, rows = sequences(case)
    need = [pages_of(n, case["page"]) for n in kv]
    children = [0] * len(kv)
    for p in parent:
        if p >= 0:
            children[p] += 1
    # the rows that move, and the pages whose number of holders changes (read and written)
    moved = sum(n for b, (n, p) in enumerate(zip(need, parent)) if p >= 0 and p != b)
    changed = sum(n for n, c in zip(need, children) if c != 1)
    fork = 8 * moved + 8 * changed + 12 * len(kv)
    if case["op"] == "fork":
        return {"bytes": fork, "flops": 0}
    more = [pages_of(n + r, case["page"]) for n, r in zip(kv, rows)]
    used = sum(n - c for n, c in zip(need, shared)) + sum(shared[::case["K"]])
    pool = used + case["spare"] + sum(more) - sum(need)
    if case["op"] == "reserve":
        # each new page's entry and count, and the pool's counts up to the last one of them (as
        # if the free ones were spread evenly), all of them to say how many are left
        new = sum(more) - sum(need)
        return {"bytes": fork + 4 * pool + 8 * new + 12 * len(kv), "flops": 0}
    return {"bytes": 8 * pool + 8 * sum(need), "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return exact_select(s)
    if op == "copy":
        n = case["n"]
        src, dst = (s["copies"][:n, i].tolist() for i in (0, 1))
        k, v = ([p.double() for p in s[name]] for name in ("k_pages", "v_pages"))
        for pages in k + v:
            pages.index_copy_(0, torch.tensor(dst, device=DEV),
                              pages.index_select(0, torch.tensor(src, device=DEV)))
        return k, v
    page, kv, refs = case["page"], s["kv_len"].tolist(), s["refs"].tolist()
    table = s["page_table"].tolist()
    used = [row[:pages_of(n, page)] for row, n in zip(table, kv)]

    def out(kv, used):
        rows = [row + old[len(row):] for row, old in zip(used, table)]
        return torch.tensor(kv, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32)

    if op == "compact":
        held = [p for p, r in enumerate(refs) if r]
        holes = [p for p in range(len(held)) if not refs[p]]
        pairs = list(zip(held[len(held) - len(holes):], holes))
        to = dict(pairs)
        new_refs = [0] * len(refs)
        for p in held:
            new_refs[to.get(p, p)] = refs[p]
        new = out(kv, [[to.get(p, p) for p in row] for row in used])[1]
        copies = s["copies"].cpu()
        if pairs:
            copies[:len(pairs)] = ints(pairs)
        return ints(new_refs), new, copies, ints([len(pairs), len(held)])
    keep = s["keep"].tolist() if op == "reserve" else [math.inf] * len(kv)
    was_kv, was = list(kv), [list(row) for row in used]
    full = [list(row) for row in table]
    for b, p in enumerate(s["parent"].tolist()):
        kv[b] = min(was_kv[p], keep[b]) if p >= 0 else 0
        used[b] = was[p][:pages_of(kv[b], page)] if p >= 0 else []
        full[b][:len(used[b])] = used[b]
    table[:] = full                                          # entries past them stay
    for rows, by in ((was, -1), (used, 1)):
        for row in rows:
            for p in row:
                refs[p] += by
    if op == "fork":
        return (*out(kv, used), ints(refs))
    start, pairs = s["row_start"].tolist(), []
    free = [p for p in reversed(range(len(refs))) if not refs[p]]
    rows = [b - a for a, b in zip(start, start[1:])]
    writers = {}
    for b, r in enumerate(rows):
        if r and kv[b] % page:
            writers.setdefault(used[b][-1], []).append(b)
    holders = {p: refs[p] for p in writers}
    for b, r in enumerate(rows):
        if r and kv[b] % page:
            p = used[b][-1]
            stays = writers[p][0] == b and len(writers[p]) == holders[p]
            if holders[p] > 1 and not stays:
                used[b][-1] = free.pop()
                pairs.append((p, used[b][-1]))
                refs[p] -= 1
                refs[used[b][-1]] = 1
        kv[b] += r
        while len(used[b]) < pages_of(kv[b], page):
            used[b].append(free.pop())
            refs[used[b][-1]] = 1
    copies = s["copies"].cpu()
    if pairs:
        copies[:len(pairs)] = ints(pairs)
    return (*out(kv, used), ints(refs), copies, ints([len(pairs), len(free)]))


def exact_select(s):
    G, K, V, N = s["G"], s["K"], s["V"], s["N"]
    score = torch.full((G, N), -math.inf, dtype=torch.float64)
    parents, tokens = (torch.full((G, N), -1, dtype=torch.int32) for _ in range(2))
    for g in range(G):
        log = s["logits"][g * K:(g + 1) * K].double()
        log = log - log.logsumexp(-1, keepdim=True)
        for k in range(K):
            if int(s["last"][g, k]) == END:
                log[k] = -math.inf
                log[k, END] = 0.0
            log[k] += float(s["scores"][g, k])
        log = log.flatten()
        for i in range(N):
            best = log.max()
            if best == -math.inf:
                break
            at = int((log == best).nonzero()[0])             # the first of equals
            score[g, i], parents[g, i], tokens[g, i] = best, g * K + at // V, at % V
            log[at] = -math.inf
    return score, parents, tokens
