"""smoe_pages_fork, smoe_pages_reserve, smoe_pages_copy and smoe_pages_compact on the GPU,
against the plain definitions on the host: whole numbers, equal to the last entry."""
import random

import pytest

torch = pytest.importorskip("torch")

from pages_helpers import Pool, pages_of, random_pool  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32, BF16 = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_expert_weight_gb300 import build
    build.build()
    import bit_expert_weight_gb300.smoe as S
    S.load()
    S.device_status()
    return S


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


class OnDevice:
    """A pool's arrays, each with a guard behind it, the table and the lengths at odd places."""

    def __init__(self, p):
        S, W, P = len(p.kv), p.width, len(p.refs)
        self.buf = [torch.full((n + 40,), -77, dtype=I32, device=DEV) for n in (P, S, S * W)]
        self.refs = self.buf[0][:P]
        self.kv = self.buf[1][3:3 + S]
        self.table = self.buf[2][5:5 + S * W].view(S, W)
        self.page = p.page
        self.put(p)

    def put(self, p):
        self.refs.copy_(ints(p.refs))
        self.kv.copy_(ints(p.kv))
        self.table.copy_(ints(p.table).view_as(self.table))

    @property
    def pool(self):
        return self.refs, self.kv, self.table, self.page

    def check(self, p):
        assert self.refs.tolist() == p.refs
        assert self.kv.tolist() == p.kv
        assert self.table.tolist() == p.table
        for b, n, first in zip(self.buf, (len(p.refs), len(p.kv), len(p.kv) * p.width), (0, 3, 5)):
            assert bool((b[:first] == -77).all()) and bool((b[first + n:] == -77).all())


def reserve(S, d, rows):
    start = [5]
    for r in rows:
        start.append(start[-1] + r)
    copies = torch.full((len(rows) + 2, 2), -5, dtype=I32, device=DEV)
    counts = torch.full((4,), -5, dtype=I32, device=DEV)
    S.pages_reserve(*d.pool, ints(start), copies[1:-1], counts[1:3])
    assert counts[0] == counts[3] == -5 and copies[0, 0] == copies[-1, 1] == -5
    return copies[1:-1].tolist(), counts[1:3].tolist()


SIZES = [  # pages, page size, sequences, table width
    (1, 16, 1, 1), (7, 16, 2, 5), (60, 32, 9, 12), (300, 16, 40, 23), (1_000, 128, 17, 70),
    (5_000, 16, 300, 40), (40_000, 256, 33, 513), (9_000, 64, 2_048, 9), (70_001, 16, 5, 4_500),
    (300_003, 16, 64, 900), (30_000, 32, 100, 700), (140_001, 64, 7, 300), (1_200_007, 16, 50, 900),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_program_of_calls(S, size):
    """Random calls one after the other on one pool, each as the definition says: every count,
    length and entry, those that are not to be touched among them."""
    P, page, n, W = size
    rng = random.Random(P + n)
    p = random_pool(P, page, n, W, seed=P)
    d = OnDevice(p)
    for step in range(14):
        what = rng.choice(["fork", "fork", "reserve", "reserve", "reserve", "compact"])
        if what == "fork":
            kind = rng.choice(["any", "own", "drop", "one"])
            parent = {"any": lambda s: rng.randint(-1, n - 1), "own": lambda s: s,
                      "drop": lambda s: s if rng.random() < 0.7 else -1,
                      "one": lambda s: 0}[kind]
            parent = [parent(s) for s in range(n)]
            keep = rng.choice([None, [rng.choice([rng.randint(-3, page * W), k, k - 1])
                                      for k in p.kv]])
            if sum(pages_of(k, page) for k in p.kv) > 200_000:
                parent = [-1 if s % 3 else q for s, q in enumerate(parent)]
            p.fork(parent, keep)
            S.pages_fork(*d.pool, ints(parent), keep=None if keep is None else ints(keep))
        elif what == "reserve":
            room = [page * W - k for k in p.kv]
            most = rng.choice([1, 1, 2 * page, page * W])
            rows = [min(r, rng.choice([0, 1, rng.randint(0, most)])) for r in room]
            want = p.reserve(rows)
            copies, counts = reserve(S, d, rows)
            if want is None:
                assert counts[0] == 0 and counts[1] < 0 and S.device_status() == -5
                assert copies == [[-5, -5]] * n
            else:
                assert counts == [len(want[0]), want[1]]
                assert copies == want[0] + [[-5, -5]] * (n - len(want[0]))
        else:
            copies = torch.full((P // 2 + 1, 2), -5, dtype=I32, device=DEV)
            counts = torch.full((3,), -5, dtype=I32, device=DEV)
            where = {}
            if rng.random() < 0.5:           # into arrays of their own
                where = dict(refs_out=torch.full((P,), 99, dtype=I32, device=DEV),
                             page_table_out=torch.full((n, W), 98, dtype=I32, device=DEV))
                before = p.copy()
            moves, held = p.compact()
            S.pages_compact(*d.pool, copies[:P // 2], counts[:2], **where)
            assert counts.tolist() == [len(moves), held, -5]
            assert copies.tolist() == moves + [[-5, -5]] * (P // 2 + 1 - len(moves))
            if where:
                d.check(before)
                assert where["refs_out"].tolist() == p.refs
                for s, row in enumerate(where["page_table_out"].tolist()):
                    k = pages_of(p.kv[s], page)
                    assert row[:k] == p.table[s][:k] and row[k:] == [98] * (W - k)
                d.refs.copy_(where["refs_out"])
                d.table.copy_(ints(p.table))
        d.check(p)
        assert S.device_status() == 0


def test_all_beams_write_apart(S):
    """2,048 sequences that share their last pages, 1 to 300 to a page."""
    rng = random.Random(1)
    p = Pool(6_000, 16, 2_048, 3)
    s = 0
    while s < 2_048:
        page, keys = p.refs.index(0), rng.randint(1, 47)
        n = min(2_048 - s, rng.choice([1, 2, 5, 300]))
        pages = list(range(page, page + pages_of(keys, 16)))
        for t in range(s, s + n):
            p.kv[t], p.table[t][:len(pages)] = keys, pages
        for q in pages:
            p.refs[q] = n + (rng.random() < 0.1)     # now and then another holder
        s += n
    order = list(range(2_048))
    rng.shuffle(order)
    p.kv, p.table = [p.kv[t] for t in order], [p.table[t] for t in order]
    for rows in ([1] * 2_048, [rng.randint(0, 1) for _ in range(2_048)]):
        q = p.copy()
        d = OnDevice(q)
        want = q.reserve(rows)
        copies, counts = reserve(S, d, rows)
        assert counts == [len(want[0]), want[1]] and copies[:counts[0]] == want[0]
        d.check(q)
    assert S.device_status() == 0


def test_not_enough_pages(S):
    p = Pool(10, 16, 3, 600)
    p.reserve([40, 16, 1])
    d = OnDevice(p)
    for rows, short in (([0, 96, 0], -1), ([9_000, 0, 400], None), ([8, 0, 0], 5)):
        copies, counts = reserve(S, d, rows)
        need = sum(pages_of(k + r, 16) - pages_of(k, 16) for k, r in zip(p.kv, rows))
        assert counts == [0, 5 - need] and (short is None or counts[1] == short)
        assert S.device_status() == (-5 if counts[1] < 0 else 0)
        if counts[1] >= 0:
            p.reserve(rows)
        d.check(p)
    # far more than the pool
    wide = Pool(10, 16, 2_000, 1)
    d = OnDevice(wide)
    table = torch.zeros(2_000, 1 << 16, dtype=I32, device=DEV)
    counts, copies = ints([0, 0]), torch.zeros(2_000, 2, dtype=I32, device=DEV)
    start = torch.arange(2_001, device=DEV, dtype=I32)
    for rows, left in ((0, 10), (1 << 20, 10 - 2_000 * 65_536)):
        S.pages_reserve(d.refs, d.kv, table, 16, start * rows, copies, counts)
        assert counts.tolist() == [0, left] and S.device_status() == (-5 if left < 0 else 0)
    d.check(wide)


def test_bad_batches_are_recorded_and_change_nothing(S):
    p = Pool(50, 16, 4, 6)
    p.reserve([20, 16, 33, 0])
    d = OnDevice(p)
    ok = [0, 1, 2, 3]

    def recorded(kv=None, table=None, refs=None, call=None):
        q = p.copy()
        if kv:
            q.kv[kv[0]] = kv[1]
        if table:
            q.table[table[0]][table[1]] = table[2]
        if refs:
            q.refs[refs[0]] = refs[1]
        d.put(q)
        call()
        assert S.device_status() == -5 and S.device_status() == 0
        d.check(q)

    fork = lambda parent: lambda: S.pages_fork(*d.pool, ints(parent))  # noqa: E731
    for parent in ([0, 1, 2, 4], [-2, 1, 2, 3], [0, 1 << 30, 2, 3]):
        recorded(call=fork(parent))
    for kv in ((1, -1), (1, 97), (3, 2 ** 31 - 1), (0, -2 ** 31)):
        recorded(kv=kv, call=fork(ok))

    def res(rows):
        def call():
            copies, counts = reserve(S, d, rows)
            assert counts == [0, -1] and copies == [[-5, -5]] * 4
        return call
    for rows in ([0, -1, 5, 0], [0, 0, 64, 0], [0, 0, 0, 97]):
        recorded(call=res(rows))
    for kv in ((1, -1), (1, 97), (3, 2 ** 31 - 1)):
        recorded(kv=kv, call=res([1, 1, 1, 1]))
    for table in ((0, 1, 50), (0, 1, -1), (2, 2, 2 ** 31 - 1)):
        recorded(table=table, call=res([1, 1, 1, 1]))
    recorded(refs=(1, 0), call=res([1, 1, 1, 1]))          # nobody holds a last page


def test_fork_records_entries_of_no_page(S):
    p = Pool(50, 16, 3, 6)
    p.reserve([40, 16, 0])
    p.table[0][1] = 50
    d = OnDevice(p)
    S.pages_fork(*d.pool, ints([-1, 1, 1]))
    assert S.device_status() == -5
    assert d.kv.tolist() == [0, 16, 16] and d.refs.tolist()[:4] == [0, 1, 0, 2]
    assert d.refs.tolist()[4:] == [0] * 46


def test_compact_records_bad_rows(S):
    p = Pool(50, 16, 4, 6)
    p.reserve([16, 40, 33, 20])
    p.fork([-1, 1, 2, 3])
    p.table[1][0] = -1
    p.table[2][1] = 40                       # a page that nobody holds
    d = OnDevice(p)
    d.kv[3] = 97
    copies, counts = torch.zeros(25, 2, dtype=I32, device=DEV), ints([0, 0])
    S.pages_compact(*d.pool, copies, counts)
    assert S.device_status() == -5
    assert counts.tolist() == [1, 8] and copies[0].tolist() == [8, 0]
    want = [list(r) for r in p.table]
    assert d.table.tolist() == want          # (page 8 is of sequence 3, whose length is wrong)
    assert d.refs.tolist() == [1] * 8 + [0] * 42


@pytest.mark.parametrize("P", [40, 140_003])   # by one launch, by four
@pytest.mark.parametrize("count", [0, -1, -3, -(2 ** 30)])
@pytest.mark.parametrize("apart", [False, True])
def test_compact_of_free_pages_below_zero(S, P, count, apart):
    """An entry that names a page which nobody holds stays and is recorded, whatever is in its count."""
    p = Pool(P, 16, 2, 4)
    p.kv, p.table = [48, 30], [[1, 7, 9, -9], [3, 12, -9, -9]]     # page 9 has no holder
    p.refs = [count] * P
    for q in (1, 3, 7, 12):
        p.refs[q] = 1
    d = OnDevice(p)
    out = dict(refs_out=torch.full((P,), 99, dtype=I32, device=DEV),
               page_table_out=torch.full((2, 4), -9, dtype=I32, device=DEV)) if apart else {}
    copies = torch.full((P // 2, 2), -5, dtype=I32, device=DEV)
    counts = torch.zeros(2, dtype=I32, device=DEV)
    S.pages_compact(*d.pool, copies, counts, **out)
    assert counts.tolist() == [2, 4] and copies[:3].tolist() == [[7, 0], [12, 2], [-5, -5]]
    refs, table = out.get("refs_out", d.refs).tolist(), out.get("page_table_out", d.table).tolist()
    assert refs[:4] == [1] * 4 and all(r <= 0 for r in refs[4:])
    assert table == [[1, 0, 9, -9], [3, 2, -9, -9]]
    assert S.device_status() == -5


def test_no_sequences_and_full_pools(S):
    p = Pool(400, 16, 1, 400)
    p.reserve([400 * 16])
    d = OnDevice(p)
    copies, counts = torch.zeros(200, 2, dtype=I32, device=DEV), ints([5, 5])
    S.pages_compact(*d.pool, copies, counts)
    assert counts.tolist() == [0, 400]
    d.check(p)
    assert reserve(S, d, [0])[1] == [0, 0]
    empty = (d.refs, d.kv[:0], d.table, 16)
    S.pages_compact(*empty, copies, counts)
    assert counts.tolist() == [0, 400]
    S.pages_reserve(*empty, ints([7]), copies, counts)
    assert counts.tolist() == [0, 0]
    S.pages_fork(*empty, ints([]))
    p.fork([-1])
    S.pages_fork(*d.pool, ints([-1]))
    S.pages_compact(*d.pool, copies, counts)
    assert counts.tolist() == [0, 0]
    d.check(p)
    assert S.device_status() == 0


def test_tables_of_no_columns(S):
    p = Pool(20, 16, 3, 0)
    d = OnDevice(p)
    S.pages_fork(*d.pool, ints([2, -1, 0]))
    assert reserve(S, d, [0, 0, 0]) == ([[-5, -5]] * 3, [0, 20])
    S.pages_compact(*d.pool, torch.zeros(10, 2, dtype=I32, device=DEV), ints([0, 0]))
    assert S.device_status() == 0
    assert reserve(S, d, [0, 1, 0]) == ([[-5, -5]] * 3, [0, -1]) and S.device_status() == -5
    d.check(p)


def test_tables_past_32_bits(S):
    """The last rows' entries are more than 2^31 entries from the first."""
    n, W, P = 1_100, 2_000_000, 300
    table = torch.full((n, W), -9, dtype=I32, device=DEV)
    refs, kv = torch.zeros(P, dtype=I32, device=DEV), torch.zeros(n, dtype=I32, device=DEV)
    start = torch.zeros(n + 1, dtype=I32, device=DEV)
    start[1:] += 3                            # rows of the first and of the last two sequences
    start[n - 1:] += 40
    start[n:] += 30
    copies, counts = torch.zeros(n, 2, dtype=I32, device=DEV), ints([0, 0])
    S.pages_reserve(refs, kv, table, 16, start, copies, counts)
    assert counts.tolist() == [0, P - 6]
    assert table[0, :2].tolist() == [0, -9]
    assert table[n - 2, :4].tolist() == [1, 2, 3, -9] and table[n - 1, :3].tolist() == [4, 5, -9]
    parent = torch.arange(n, dtype=I32, device=DEV)
    parent[0], parent[n - 1] = n - 2, -1
    S.pages_fork(refs, kv, table, 16, parent)
    assert table[0, :4].tolist() == [1, 2, 3, -9] and refs[:7].tolist() == [0, 2, 2, 2, 0, 0, 0]
    moves = torch.zeros(P // 2, 2, dtype=I32, device=DEV)
    S.pages_compact(refs, kv, table, 16, moves, counts)
    assert counts.tolist() == [1, 3] and moves[0].tolist() == [3, 0]
    assert table[n - 2, :4].tolist() == [1, 2, 0, -9] and table[0, :4].tolist() == [1, 2, 0, -9]
    assert S.device_status() == 0


def test_large_pools(S):
    """70 million pages: the free ones far behind, and a compaction of half of them."""
    P, page = 70_000_001, 16
    refs = torch.ones(P, dtype=I32, device=DEV)
    free = [5, 12_345_678, P - 3, P - 1]
    refs[free] = 0
    kv, table = ints([0, 0]), torch.full((2, 9), -9, dtype=I32, device=DEV)
    copies, counts = torch.zeros(P // 2, 2, dtype=I32, device=DEV), ints([0, 0])
    S.pages_reserve(refs, kv, table, page, ints([0, 17, 50]), copies, counts)
    assert counts.tolist() == [0, -1] and S.device_status() == -5 and kv.tolist() == [0, 0]
    S.pages_reserve(refs, kv, table, page, ints([0, 17, 40]), copies, counts)
    assert counts.tolist() == [0, 0] and bool((refs == 1).all())
    assert table[:, :3].tolist() == [free[:2] + [-9], free[2:] + [-9]]
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    refs.copy_(torch.randint(0, 3, (P,), generator=g, device=DEV, dtype=I32))
    refs[free] = 1
    was = refs.clone()
    held = (was > 0).nonzero()[:, 0]
    n = held.numel()
    source = held[held >= n]
    target = (was[:n] <= 0).nonzero()[:, 0]
    for out in (None, torch.full((P,), 9, dtype=I32, device=DEV)):
        refs.copy_(was)
        before = table.clone()
        into = torch.empty_like(table) if out is not None else None
        S.pages_compact(refs, kv, table if out is not None else before, page, copies, counts,
                        refs_out=out, page_table_out=into)
        assert S.device_status() == 0 and counts.tolist() == [source.numel(), n]
        m = copies[:source.numel()].long()
        assert torch.equal(m[:, 0], source) and torch.equal(m[:, 1], target)
        want = was.clone()
        want[target] = was[source]
        want[n:] = 0
        assert torch.equal(want, refs if out is None else out)
        now = (before if out is None else into)[:, :2]
        moved = {int(a): int(b) for a, b in zip(source[-3:], target[-3:])}
        assert now[0, 0] == 5 and now[1, 1] == moved.get(P - 1, P - 1)
        assert now[0, 1] == (12_345_678 if 12_345_678 < n else None)


# --------------------------------------------------------------- copies

@pytest.mark.parametrize("P, n, W, chance", [
    (140_003, 40, 1_500, 0.5), (430_000, 200, 1_000, 0.5), (524_288, 2_000, 130, 0.3),
    (1_700_011, 100, 9_000, 0.5), (5_000_000, 64, 50_000, 0.1), (9_000_001, 2_048, 4_000, 0.05)], ids=str)
def test_many_pages_given_at_once(S, P, n, W, chance):
    """Almost all that a large pool has left, given away by one call, time after time: each
    page of the pool is looked at while others are given."""
    gen = torch.Generator(device=DEV).manual_seed(P)
    for turn in range(6):
        refs = (torch.rand(P, device=DEV, generator=gen) < chance).to(I32)
        refs[:(turn * P) // 7] *= turn % 2
        free = (refs <= 0).nonzero()[:, 0]
        need = torch.randint(0, 2 * min(W, len(free) // n), (n,), device=DEV, generator=gen).clamp(max=W)
        need = (need * min(1.0, len(free) / max(1, int(need.sum())))).long()
        start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), need.cumsum(0)])
        table = torch.full((n, W), -9, dtype=I32, device=DEV)
        kv = torch.zeros(n, dtype=I32, device=DEV)
        copies = torch.full((n, 2), -5, dtype=I32, device=DEV)
        counts = torch.full((2,), -5, dtype=I32, device=DEV)
        want_refs, total = refs.clone(), int(start[-1])
        want_refs[free[:total]] = 1
        own = torch.arange(W, device=DEV) < need[:, None]
        want = table.clone()
        want[own] = free[:total].to(I32)
        S.pages_reserve(refs, kv, table, 16, (16 * start).to(I32), copies, counts)
        assert counts.tolist() == [0, len(free) - total], turn
        assert torch.equal(kv, (16 * need).to(I32)) and bool((copies == -5).all())
        assert torch.equal(table, want), turn
        assert torch.equal(refs, want_refs), turn
    assert S.device_status() == 0


def caches(layers, P, Hkv, page, D, joined, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def bits(*shape):                        # any bits at all, NaNs among them
        return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device=DEV,
                             dtype=torch.int16).view(BF16)

    if joined:
        both = [bits(P, 2, Hkv, page, D) for _ in range(layers)]
        return [b[:, 0] for b in both], [b[:, 1] for b in both]
    return [bits(P, Hkv, page, D) for _ in range(layers)], [bits(P, Hkv, page, D)
                                                            for _ in range(layers)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("layers, n, most, P, Hkv, page, D, joined", [
    (1, 1, 1, 2, 1, 16, 64, False), (1, 0, 4, 9, 2, 16, 64, False), (3, 5, 5, 11, 3, 32, 128, True),
    (2, 7, 40, 30, 5, 16, 64, True), (128, 3, 9, 8, 1, 16, 64, False),
    (94, 20, 25, 50, 4, 16, 128, True), (1, 300, 301, 700, 8, 256, 128, False),
    (2, 40, 64, 90, 7, 64, 64, False), (1, 2, 3, 6, 33, 128, 128, True),
], ids=str)
def test_copy(S, layers, n, most, P, Hkv, page, D, joined):
    k, v = caches(layers, P, Hkv, page, D, joined)
    g = torch.Generator(device=DEV)
    g.manual_seed(n)
    ids = torch.randperm(P, generator=g, device=DEV)[:2 * n].to(I32).view(-1, 2)
    if n > 2:
        ids[1, 0] = ids[0, 0]                # one page to two others
    copies = torch.full((most, 2), 1 << 29, dtype=I32, device=DEV)
    copies[:n] = ids
    want = [[x.clone() for x in xs] for xs in (k, v)]
    for xs in want:
        for x in xs:
            x[ids[:, 1].long()] = x[ids[:, 0].long()]
    one = layers == 1
    S.pages_copy(k[0] if one else k, v[0] if one else v, copies, ints([n, 77]))
    assert S.device_status() == 0
    for xs, ws in zip((k, v), want):
        assert all(same_bits(a, b) for a, b in zip(xs, ws))


def test_copy_records_bad_pages_and_counts(S):
    k, v = caches(2, 8, 2, 16, 64, False)
    want = [[x.clone() for x in xs] for xs in (k, v)]
    for xs in want:
        for x in xs:
            x[3], x[5] = x[1], x[2]
    pairs = [[1, 3], [8, 4], [0, -1], [0, 8], [-1, 6], [2 ** 31 - 1, 7], [2, 5]]
    S.pages_copy(k, v, ints(pairs), ints([7]))
    assert S.device_status() == -5 and S.device_status() == 0
    for xs, ws in zip((k, v), want):
        assert all(same_bits(a, b) for a, b in zip(xs, ws))
    for count in (-1, -2 ** 31, 3, 2 ** 31 - 1):           # two pairs at most
        S.pages_copy(k, v, ints([[1, 3], [2, 5]]), ints([count]))
        assert S.device_status() == -5 and S.device_status() == 0
        for xs, ws in zip((k, v), want):
            assert all(same_bits(a, b) for a, b in zip(xs, ws))


def test_copies_past_32_bits(S):
    """Pages that are more than 2^31 elements from the first."""
    P = 2_200_000
    k = torch.zeros(P, 1, 16, 64, dtype=BF16, device=DEV)
    v = torch.zeros(P, 1, 16, 64, dtype=BF16, device=DEV)
    (a,), (b,) = caches(1, 3, 1, 16, 64, False)
    k[:3], v[:3] = a, b
    S.pages_copy(k, v, ints([[0, P - 1], [2, P - 2]]), ints([2]))
    S.pages_copy(k, v, ints([[P - 1, 7]]), ints([1]))
    assert S.device_status() == 0
    for x, y in ((k, a), (v, b)):
        assert same_bits(x[P - 1], y[0]) and same_bits(x[P - 2], y[2]) and same_bits(x[7], y[0])
        assert not bool(x[8:P - 2].view(torch.int16).any())


def test_captured_steps(S):
    """Fork, reserve and copy captured together and replayed with other parents and rows."""
    P, page, n, W = 400, 16, 12, 20
    rng = random.Random(3)
    p = random_pool(P, page, n, W, seed=4)
    p.kv = [min(k, page * (W // 2)) for k in p.kv]
    p.fork(list(range(n)))
    used = [0] * P
    for s in range(n):
        for q in p.used(s):
            used[q] += 1
    p.refs = used
    d = OnDevice(p)
    k, v = caches(2, P, 2, page, 64, True)
    parent, start = ints(list(range(n))), ints([0] * (n + 1))
    copies, counts = torch.zeros(n, 2, dtype=I32, device=DEV), ints([0, 0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.pages_fork(*d.pool, parent)
        S.pages_reserve(*d.pool, start, copies, counts)
        S.pages_copy(k, v, copies, counts)
    for _ in range(6):
        order = [rng.randrange(n) for _ in range(n)]
        rows = [rng.randint(0, 2) for _ in range(n)]
        parent.copy_(ints(order))
        start.copy_(ints([sum(rows[:i]) for i in range(n + 1)]))
        p.fork(order)
        pairs, left = p.reserve(rows)
        want = [x.clone() for x in k + v]
        for x in want:
            for a, b in pairs:
                x[b] = x[a]
        graph.replay()
        torch.cuda.synchronize()
        assert counts.tolist() == [len(pairs), left]
        d.check(p)
        assert all(same_bits(a, b) for a, b in zip(k + v, want))
    assert S.device_status() == 0
