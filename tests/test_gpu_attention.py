"""smoe_attention on the GPU against its 64-bit definition."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import Paged  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


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


@pytest.fixture(scope="module")
def ws(S):
    return S.attention_workspace(DEV)


def run(S, ws, p, **kw):
    return S.attention(kw.pop("q", p.q), p.k_pages, p.v_pages, p.row_start, p.kv_len,
                       p.page_table, kw.pop("max_rows", p.max_rows), ws, **kw)


# rows and keys of each sequence; query heads, kv heads, head_dim, page, window
SINGLE = [
    ([1], [1], 1, 1, 64, 16, 0),
    ([1], [16], 16, 1, 128, 16, 0),
    ([1], [17], 4, 4, 128, 16, 0),
    ([1], [777], 64, 4, 128, 16, 0),
    ([1] * 5, [127, 128, 129, 255, 257], 8, 8, 64, 32, 0),
    ([1] * 40, [(997 * i) % 1500 for i in range(40)], 24, 8, 128, 64, 0),
    ([1, 0, 1, 0], [300, 500, 0, 0], 10, 2, 128, 128, 0),
    ([1] * 3, [5000, 3, 20_011], 7, 1, 128, 256, 0),
    ([1] * 4, [100, 64, 65, 2000], 8, 2, 64, 16, 64),
    ([1] * 4, [1, 2, 130, 1000], 8, 2, 128, 16, 1),
    ([2] * 3, [2, 40, 700], 16, 2, 128, 16, 0),
    ([3, 1, 0, 5], [1, 1, 0, 3], 6, 2, 64, 16, 0),            # chunks longer than kv_len
    ([2] * 40, [(331 * i) % 1200 + 2 for i in range(40)], 32, 2, 128, 16, 0),
    ([7, 7, 0, 1], [7, 3, 300, 4000], 8, 2, 64, 64, 64),
    ([6, 2], [700, 5], 5, 1, 128, 32, 200),
]
CHUNKS = [
    ([5] * 6, [5, 6, 130, 131, 997, 4000], 32, 8, 128, 32, 0),
    ([16], [16], 16, 2, 128, 64, 0),
    ([33], [33], 4, 4, 64, 64, 0),
    ([127, 128, 129], [127, 128, 129], 8, 2, 128, 16, 0),
    ([300, 1, 0, 45], [300, 700, 90, 1000], 16, 1, 128, 64, 0),
    ([200, 77], [1111, 77], 10, 2, 64, 32, 0),
    ([513], [513], 3, 1, 128, 128, 0),
    ([100, 200], [600, 200], 14, 2, 128, 64, 37),
    ([700], [900], 40, 8, 64, 16, 128),
    ([129, 300], [100, 5], 6, 2, 128, 64, 0),                 # chunks longer than kv_len
    ([40], [260], 128, 1, 128, 256, 0),
    ([1] * 30 + [260], [(619 * i) % 900 + 1 for i in range(30)] + [1500], 64, 4, 128, 64, 0),
]


@pytest.mark.parametrize("case", SINGLE + CHUNKS, ids=str)
def test_attention(S, ws, case):
    rows, kv, Hq, Hkv, D, page, window = case
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=len(rows) + page)
    out = run(S, ws, p, window=window)
    assert S.device_status() == 0
    p.check(out, True, window)
    assert torch.equal(out, run(S, ws, p, window=window))


@pytest.mark.parametrize("case", [SINGLE[3], SINGLE[8], CHUNKS[0], CHUNKS[4]], ids=str)
def test_attention_fp32_out_views_and_scale(S, ws, case):
    rows, kv, Hq, Hkv, D, page, window = case
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=3, joined=True)
    wide = torch.zeros(p.T, Hq + 3, D, dtype=BF16, device=DEV)
    q = wide[:, 2:2 + Hq]
    q.copy_(p.q)
    out = torch.full((p.T, Hq + 1, D + 8), 9.0, device=DEV)
    run(S, ws, p, q=q, out=out[:, 1:, :D], window=window, scale=0.3)
    assert S.device_status() == 0
    p.check(out[:, 1:, :D], True, window, scale=0.3)
    assert bool((out[:, 0] == 9.0).all()) and bool((out[..., D:] == 9.0).all())


@pytest.mark.parametrize("case", [
    # more sequences than a CTA has threads, and as many as a batch may have
    ([1] * 600, [(37 * i) % 130 for i in range(600)], 4, 2, 64, 16, 0),
    ([1] * 2048, [(53 * i) % 90 + 1 for i in range(2048)], 8, 1, 128, 16, 0),
    ([1] * 690 + [40] * 10, [(29 * i) % 200 + 40 for i in range(700)], 8, 2, 64, 32, 0),
    ([2, 0, 20] * 682, [(31 * i) % 60 + 20 for i in range(2046)], 4, 1, 128, 16, 0),
    # more tiles than a CTA has threads
    ([4500, 1], [4500, 300], 32, 1, 64, 256, 0),
    # few rows over many keys: items cut into many parts
    ([20, 3], [60_001, 35_000], 16, 2, 128, 128, 0),
    ([70], [50_000], 2, 1, 64, 64, 40_000),
], ids=lambda c: f"{len(c[0])} sequences, rows {max(c[0])}, keys {max(c[1])}")
def test_wide_batches(S, ws, case):
    rows, kv, Hq, Hkv, D, page, window = case
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=len(rows))
    out = run(S, ws, p, window=window)
    assert S.device_status() == 0
    p.check(out, True, window)
    assert torch.equal(out, run(S, ws, p, window=window))


@pytest.mark.parametrize("max_rows", [1, 3, 500])
def test_idle_batch(S, ws, max_rows):
    """No sequence has a row: nothing is written, and the workspace stays usable."""
    p = Paged([0, 0, 0], [40, 0, 7], 8, 2, 128, 16, DEV)
    q = torch.zeros(5, 8, 128, dtype=BF16, device=DEV)
    out = torch.full_like(q, 3.0)
    run(S, ws, p, q=q, out=out, max_rows=max_rows)
    assert S.device_status() == 0 and bool((out == 3.0).all())
    assert not bool(ws[:4096].any())


def test_large_scores(S, ws):
    """Scores far apart, and growing along the keys: each new maximum rescales."""
    for rows, kv, D in (([1, 1], [900, 333], 128), ([150, 70], [900, 333], 128),
                        ([64], [2000], 64)):
        p = Paged(rows, kv, 8, 2, D, 16, DEV, seed=8)
        for b, n in enumerate(kv):
            i = torch.arange(n, device=DEV)
            pg = p.page_table[b, i // 16].long()
            p.k_pages[pg, :, i % 16] = (p.k_pages[pg, :, i % 16].float() *
                                        (0.05 + i / n)[:, None, None] * 4).to(BF16)
        out = run(S, ws, p)
        p.check(out, True)


def test_later_keys_do_not_reach_earlier_rows(S, ws):
    """A row depends on the keys up to its own alone, to the bit."""
    p = Paged([200], [500], 8, 2, 128, 64, DEV, seed=4)
    ref = run(S, ws, p)
    i = torch.arange(400, 500, device=DEV)
    pg = p.page_table[0, i // 64].long()
    for pages in (p.k_pages, p.v_pages):
        pages[pg, :, i % 64] = 1e4
    out = run(S, ws, p)
    assert torch.equal(out[:100], ref[:100]) and not torch.equal(out[100:], ref[100:])


def test_rows_of_no_sequence_are_left_alone(S, ws):
    p = Paged([1, 20], [30, 60], 8, 2, 64, 16, DEV)
    q = torch.cat([p.q, torch.full((9, 8, 64), math.nan, dtype=BF16, device=DEV)])
    out = torch.full_like(q, 5.0)
    run(S, ws, p, q=q, out=out)
    assert S.device_status() == 0
    p.check(out[:21], True, q=q)
    assert bool((out[21:] == 5.0).all())


@pytest.mark.parametrize("rows", [[1, 1], [40, 50]], ids=str)
@pytest.mark.parametrize("fault", ["page_high", "page_negative", "past_table", "rows", "start"])
def test_attention_records_faults(S, ws, rows, fault):
    """A bad index is caught by the kernel's own checks: the host reads the fault once, the
    other sequence's output is right."""
    p = Paged(rows, [200, 300], 8, 2, 128, 16, DEV, seed=6)
    table, starts, lens, most = p.page_table.clone(), p.row_start.clone(), p.kv_len.clone(), 50
    if fault == "page_high":
        table[0, 3] = p.pool
    elif fault == "page_negative":
        table[0, 3] = -2 ** 31
    elif fault == "past_table":
        lens[0] = 16 * table.shape[1] + 1
    elif fault == "rows":
        p = Paged([rows[0] + 70, rows[1]], [200, 300], 8, 2, 128, 16, DEV, seed=6)
        table, starts, lens, most = p.page_table, p.row_start, p.kv_len, max(rows)
    else:
        starts[0] = -1
    out = S.attention(p.q, p.k_pages, p.v_pages, starts, lens, table, most, ws)
    assert S.device_status() == -5 and S.device_status() == 0
    n0 = p.rows[0]
    p.rows, p.kv, p.page_table = p.rows[1:], p.kv[1:], p.page_table[1:]
    p.check(out[n0:], True, q=p.q[n0:])
    ws.zero_()


def test_far_pages(S, ws):
    """Keys past 2^31 elements of the pool."""
    Hkv, page, D = 8, 256, 128
    pool = 2 ** 31 // (Hkv * page * D) + 3
    for rows in ([1], [30]):
        p = Paged(rows, [300], 16, Hkv, D, page, DEV)
        k = torch.zeros(pool, Hkv, page, D, dtype=BF16, device=DEV)
        v = torch.zeros(pool, Hkv, page, D, dtype=BF16, device=DEV)
        table = torch.tensor([[pool - 1, pool - 2]], dtype=torch.int32, device=DEV)
        for i in range(2):
            k[pool - 1 - i] = p.k_pages[p.page_table[0, i]]
            v[pool - 1 - i] = p.v_pages[p.page_table[0, i]]
        ref = run(S, ws, p)
        out = S.attention(p.q, k, v, p.row_start, p.kv_len, table, p.max_rows, ws)
        assert torch.equal(out, ref)
        del k, v
        torch.cuda.empty_cache()


def test_graph_and_streams(S, ws):
    """One captured graph serves a shrinking and a growing batch; another stream with a
    workspace of its own gives the same bits."""
    p = Paged([1] * 12, [50 + 97 * i for i in range(12)], 16, 2, 128, 16, DEV, seed=2)
    ref = run(S, ws, p)
    side, ws2 = torch.cuda.Stream(), S.attention_workspace(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = run(S, ws2, p)
    side.synchronize()
    assert torch.equal(out, ref)
    lens, start = p.kv_len.clone(), p.row_start.clone()
    q = p.q.clone()
    out = torch.empty_like(ref)
    graph = torch.cuda.CUDAGraph()
    S.attention(q, p.k_pages, p.v_pages, start, lens, p.page_table, 1, ws, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        S.attention(q, p.k_pages, p.v_pages, start, lens, p.page_table, 1, ws, out=out)
    out.zero_()
    graph.replay()
    assert torch.equal(out, ref)
    start[5:] = 4                      # the last 8 sequences sit out
    out.fill_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    p4 = Paged(p.rows[:4], p.kv[:4], 16, 2, 128, 16, DEV)
    p4.k_pages, p4.v_pages, p4.page_table = p.k_pages, p.v_pages, p.page_table
    p4.check(out[:4], True, q=q[:4])
    assert bool((out[4:] == 1.0).all())
    start.copy_(p.row_start)
    lens -= 7
    graph.replay()
    torch.cuda.synchronize()
    p.kv = [n - 7 for n in p.kv]
    p.check(out, True, q=q)
    assert S.device_status() == 0
