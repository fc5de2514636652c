"""smoe_rope and smoe_kv_append on the GPU against their 64-bit definitions."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import Paged, UBF, turned, turned_bound  # noqa: E402
from test_decoder_args import freqs  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


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


def freq64(R, theta=1e4, **kw):
    return torch.tensor(freqs(R, theta, **kw), dtype=torch.float64, device=DEV)


def randn(*shape, seed=0, dtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def inside(got, ref, tol):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{int(bad.sum())} values off, first {bad.nonzero()[0].tolist()}: "
                           f"{float(got[bad][0])} for {float(ref[bad][0])}")


ROPE = [  # T, H, D, R, interleaved, dtype, norm, positions
    (1, 1, 128, 128, False, BF16, False, "near"),
    (1, 64, 128, 128, False, BF16, True, "far"),
    (37, 5, 64, 64, True, F32, False, "far"),
    (129, 9, 128, 64, False, F32, True, "near"),
    (33, 3, 128, 32, True, BF16, True, "far"),
    (5, 40, 64, 24, False, BF16, False, "far"),
    (17, 2, 256, 256, False, F32, True, "negative"),
    (9, 7, 96, 96, True, BF16, True, "negative"),
    (3, 2, 8, 8, False, F32, False, "edge"),
    (4, 11, 80, 40, False, F32, True, "edge"),
    (1000, 33, 128, 128, False, BF16, True, "far"),
]


def positions_of(kind, T):
    i = torch.arange(T)
    p = {"near": i, "far": i * 7919 % 65_536 + 983_040, "negative": -3 * i - 1,
         "edge": torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1])[:T]}[kind]
    return p.to(torch.int32).to(DEV)


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(S, case):
    T, H, D, R, inter, dtype, norm, kind = case
    table, scale = S.rope_table(R, 1e4, device=DEV)
    x = randn(T, H, D, seed=T, dtype=dtype)
    w = randn(D, seed=1, dtype=BF16) if norm else None
    pos = positions_of(kind, T)
    got = S.rope(x, pos, table, scale, interleaved=inter, norm_w=w)
    ref, size = turned(x, pos, freq64(R), scale, inter, w)
    inside(got, ref, turned_bound(ref, size, dtype))


def test_rope_scaled_table_strides_and_in_place(S):
    table, scale = S.rope_table(64, 1e6, "parts", 16.0, device=DEV)
    assert scale > 1.2
    wide = randn(50, 12, 128, seed=3)                # rows of one projection
    keep = wide.clone()
    x = wide[:, 3:9]
    pos = positions_of("far", 50)
    f = freq64(64, 1e6, kind="parts", factor=16.0)
    ref, size = turned(x, pos, f, scale, False)
    out = torch.full((50, 14, 136), 7.0, device=DEV)[:, 2:8, :128]
    S.rope(x, pos, table, scale, out=out)
    assert torch.equal(wide, keep)
    inside(out, ref, turned_bound(ref, size, F32))
    S.rope(x, pos, table, scale, out=x)              # in place: the same bits
    assert torch.equal(x, out)
    assert torch.equal(wide[:, :3], keep[:, :3]) and torch.equal(wide[:, 9:], keep[:, 9:])


def test_rope_back(S):
    """The rotation by negative positions undoes it."""
    table, scale = S.rope_table(128, 1e4, device=DEV)
    x = randn(40, 4, 128, seed=5)
    pos = positions_of("far", 40)
    back = S.rope(S.rope(x, pos, table), -pos, table)
    ref, size = turned(x, torch.zeros_like(pos), freq64(128), 1.0, False)
    inside(back, ref, 2 * 1.5 * turned_bound(ref, size, F32))  # sizes grow by sqrt 2 at most


def test_rope_on_another_stream(S):
    table, _ = S.rope_table(128, 1e4, device=DEV)
    x, pos = randn(2000, 32, 128, seed=6), positions_of("far", 2000)
    ref = S.rope(x, pos, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = S.rope(x, pos, table, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    with torch.cuda.stream(side):
        z = S.rope(x, pos, table)
    side.synchronize()
    assert torch.equal(z, ref)


APPEND = [  # rows, kv, Hq, Hkv, D, R, page, interleaved, dtype, norm
    ([1], [1], 8, 1, 128, 128, 16, False, BF16, False),
    ([1] * 40, [(37 * i) % 300 + 1 for i in range(40)], 16, 4, 128, 128, 16, False, BF16, True),
    ([5, 0, 31, 1, 64], [5, 9, 100, 1, 65], 6, 2, 64, 32, 32, True, F32, True),
    ([130, 17], [257, 17], 10, 5, 128, 64, 256, False, F32, False),
    ([0, 0, 3, 0, 1, 0], [4, 0, 3, 7, 2, 0], 3, 3, 64, 64, 64, True, BF16, False),
    ([7, 2], [4, 1], 4, 2, 128, 128, 16, False, BF16, False),     # more rows than keys
]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("joined", [False, True])
def test_append(S, case, joined):
    rows, kv, Hq, Hkv, D, R, page, inter, dtype, norm = case
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=len(rows), joined=joined)
    T = p.T
    qkv = randn(T, Hq + 2 * Hkv, D, seed=2, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    wq, wk = (randn(D, seed=s, dtype=BF16) if norm else None for s in (3, 4))
    table, _ = S.rope_table(R, 1e4, device=DEV)
    k0, v0 = p.k_pages.clone(), p.v_pages.clone()
    got = S.kv_append(q, k, v, p.k_pages, p.v_pages, p.row_start, p.kv_len, p.page_table, table,
                      interleaved=inter, q_norm=wq, k_norm=wk)
    assert S.device_status() == 0
    index = torch.cat([torch.arange(n - r, n) for r, n in zip(rows, kv)]).to(DEV)
    ref, size = turned(q, index, freq64(R), 1.0, inter, wq)
    inside(got, ref, turned_bound(ref, size, BF16))
    ref, size = turned(k, index, freq64(R), 1.0, inter, wk)
    tol = turned_bound(ref, size, BF16)
    owner = torch.cat([torch.full((r,), b) for b, r in enumerate(rows)]).to(DEV)
    stored = (index >= 0).nonzero()[:, 0]
    pg = p.page_table[owner[stored], index[stored] // page].long()
    at = index[stored] % page
    inside(p.k_pages[pg, :, at], ref[stored], tol[stored])
    assert torch.equal(p.v_pages[pg, :, at], v[stored].to(BF16))
    # every other slot keeps its bits
    k0[pg, :, at], v0[pg, :, at] = p.k_pages[pg, :, at], p.v_pages[pg, :, at]
    for old, new in ((k0, p.k_pages), (v0, p.v_pages)):
        assert torch.equal(old.view(torch.int16), new.view(torch.int16))


def test_append_options(S):
    """No rotation, own positions, no queries, queries in place."""
    rows, kv = [3, 20], [40, 20]
    p = Paged(rows, kv, 4, 2, 128, 16, DEV)
    q, k, v = (randn(p.T, h, 128, seed=s, dtype=BF16) for h, s in ((4, 1), (2, 2), (2, 3)))
    where = (p.k_pages, p.v_pages, p.row_start, p.kv_len, p.page_table)
    assert torch.equal(S.kv_append(q, k, v, *where), q)
    i = torch.arange(37, 40, device=DEV)
    pg = p.page_table[0, i // 16].long()
    assert torch.equal(p.k_pages[pg, :, i % 16], k[:3])
    table, _ = S.rope_table(128, 1e4, device=DEV)
    pos = positions_of("far", p.T)
    ref = S.rope(k, pos, table)
    assert S.kv_append(None, k, v, *where, table, positions=pos) is None
    assert torch.equal(p.k_pages[pg, :, i % 16], ref[:3])
    ref = S.rope(q, pos, table)
    S.kv_append(q, k, v, *where, table, positions=pos, q_out=q)
    assert torch.equal(q, ref)
    assert S.device_status() == 0


def test_append_ignores_rows_of_no_sequence(S):
    p = Paged([2, 1], [5, 8], 4, 2, 64, 16, DEV)
    q, k, v = (randn(10, h, 64, seed=s, dtype=BF16) for h, s in ((4, 1), (2, 2), (2, 3)))
    k0 = p.k_pages.clone()
    out = torch.full_like(q, 3.0)
    S.kv_append(q, k, v, p.k_pages, p.v_pages, p.row_start, p.kv_len, p.page_table, q_out=out)
    assert torch.equal(out[:3], q[:3]) and bool((out[3:] == 3.0).all())
    assert int((k0.view(torch.int16) != p.k_pages.view(torch.int16)).any(-1).sum()) <= 3 * 2
    assert S.device_status() == 0


@pytest.mark.parametrize("fault", ["page_high", "page_negative", "past_table", "row_start"])
def test_append_records_faults(S, fault):
    """Each bad index is caught by the kernel's own checks: nothing is stored for it, the
    other sequence is stored, and the host reads the fault once."""
    p = Paged([2, 2], [20, 20], 4, 2, 64, 16, DEV)
    k, v = (randn(4, 2, 64, seed=s, dtype=BF16) for s in (2, 3))
    table, starts, lens = p.page_table.clone(), p.row_start.clone(), p.kv_len.clone()
    if fault == "page_high":
        table[0, 1] = p.pool
    elif fault == "page_negative":
        table[0, 1] = -1
    elif fault == "past_table":
        lens[0] = 16 * table.shape[1] + 2
    else:
        starts[0] = -5
    k0 = p.k_pages.clone()
    S.kv_append(None, k, v, p.k_pages, p.v_pages, starts, lens, table)
    assert S.device_status() == -5 and S.device_status() == 0
    i = torch.arange(18, 20, device=DEV)
    pg = p.page_table[1, i // 16].long()
    assert torch.equal(p.k_pages[pg, :, i % 16], k[2:])
    k0[pg, :, i % 16] = k[2:]
    assert torch.equal(k0.view(torch.int16), p.k_pages.view(torch.int16))


def test_append_far_pages(S):
    """Slots past 2^31 elements of the pool."""
    Hkv, page, D = 8, 256, 128
    per = Hkv * page * D
    pool = 2 ** 31 // per + 3
    pages = torch.zeros(pool, Hkv, page, D, dtype=BF16, device=DEV)
    table = torch.tensor([[pool - 1]], dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    lens = torch.tensor([200], dtype=torch.int32, device=DEV)
    k = randn(3, Hkv, D, seed=1, dtype=BF16)
    v = torch.zeros(2, Hkv, page, D, dtype=BF16, device=DEV)
    S.kv_append(None, k, k, pages, pages, start, lens, table)
    assert S.device_status() == 0
    assert torch.equal(pages[pool - 1, :, 197:200].transpose(0, 1), k)
    assert int(pages.view(torch.int16).any(-1).sum()) == 3 * Hkv
    del v
