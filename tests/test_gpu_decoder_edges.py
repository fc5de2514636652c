"""Edges of rope, kv_append and attention on the GPU: views whose rows overlap, row starts,
long lines of work, values and scores of large size."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import Paged, attend_bound, turned, turned_bound  # noqa: E402
from test_attn_bounds import FEW  # noqa: E402
from test_decoder_args import freqs  # noqa: E402

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


def randn(*shape, seed=0, dtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def test_inputs_whose_rows_overlap(S, ws):
    """Rows of a sliding window over one buffer: the outputs are the plain copy's, to the bit."""
    T, H, D = 5, 4, 64
    x = torch.as_strided(randn(2000, dtype=BF16), (T, H, D), (8, 64, 1))
    table, _ = S.rope_table(D, 1e4, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    out = S.rope(x, pos, table)
    assert torch.equal(out, S.rope(x.contiguous(), pos, table))
    ref, size = turned(x, pos, torch.tensor(freqs(D, 1e4), dtype=torch.float64, device=DEV), 1.0,
                       False)
    assert bool(((out.double() - ref).abs() <= turned_bound(ref, size, BF16)).all())
    p = Paged([T], [40], H, 2, D, 16, DEV)
    where = (p.k_pages, p.v_pages, p.row_start, p.kv_len, p.page_table)
    k = x[:, :2]
    assert torch.equal(S.kv_append(x, k, k, *where, table),
                       S.kv_append(x.contiguous(), k, k, *where, table))
    assert torch.equal(S.attention(x, *where, T, ws), S.attention(x.contiguous(), *where, T, ws))
    assert S.device_status() == 0


def attend_paged(S, ws, p, max_rows=None, **kw):
    return S.attention(p.q, p.k_pages, p.v_pages, p.row_start, p.kv_len, p.page_table,
                       max_rows or p.max_rows, ws, **kw)


@pytest.mark.parametrize("rows, G", [(64, 1), (300, 2), (1, 4), (6, 4)], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_values_of_large_size(S, ws, rows, G, D):
    """Values of up to 2^118 under scores that grow by 2^29 and 2^6 along the keys.  Weights
    that are relative to the largest score so far are at most 1, so that sums over 400 keys
    stay below 2^127; were they 2^29, they would not."""
    n = 400
    p = Paged([rows], [n], 2 * G, 2, D, 16, DEV, seed=5)
    i = torch.arange(n, device=DEV)
    pg, at = p.page_table[0, i // 16].long(), i % 16
    p.q.zero_()
    p.q[..., 0] = 1
    key = torch.zeros(n, 2, D, dtype=BF16, device=DEV)
    key[:, :, 0] = torch.where(i < 100, 0.0, torch.where(i < 330, 20.0, 24.0))[:, None].to(BF16)
    p.k_pages[pg, :, at] = key
    sign = randn(n, 2, D, seed=1).add(0.5).sign()
    p.v_pages[pg, :, at] = (sign * randn(n, 2, D, seed=2).abs().clamp(1, 2) * 2.0 ** 117).to(BF16)
    for dtype in (F32, BF16):
        out = attend_paged(S, ws, p, scale=1.0, out_dtype=dtype)
        assert bool(torch.isfinite(out).all())
        p.check(out, True, scale=1.0)
    assert S.device_status() == 0


@pytest.mark.parametrize("step", [9.0, 50.0])
@pytest.mark.parametrize("rows, kv, Hq, Hkv, D", [
    ([300], [2000], 2, 2, 64),
    ([300], [2000], 2, 2, 128),
    ([40, 9], [1500, 900], 16, 2, 128),
    ([20], [60_001], 16, 2, 64),            # one tile of keys for many CTAs
], ids=str)
def test_maxima_that_keep_growing(S, ws, rows, kv, Hq, Hkv, D, step):
    """Every other row's scores grow by 2^step at most 12 times along the keys, so that what
    is summed so far has to be scaled again and again; the rows between, in the same warps,
    see scores of one size and are not scaled."""
    page = 64
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=11)
    scale = math.log(2) / 4
    odd = (torch.arange(p.T, device=DEV)[:, None] + torch.arange(Hq, device=DEV)) % 2 == 1
    p.q[odd] = 0
    p.q[..., 0] = torch.where(odd, 4.0, 0.0).to(BF16)       # odd rows: the key's channel 0
    for b, n in enumerate(kv):
        i = torch.arange(n, device=DEV)
        pg, at = p.page_table[b, i // page].long(), i % page
        block = i // 64
        times = block * 12 // int(block[-1]) if n > 2000 else block.clamp(max=12)
        key = p.k_pages[pg, :, at]
        key[..., 0] = (times * step)[:, None].to(BF16)
        p.k_pages[pg, :, at] = key
        # what the rows see, in powers of two per 64 keys, of the last row
        row = sum(rows[:b + 1]) - 1
        q = p.q[row].double().view(Hkv, Hq // Hkv, D)
        s = torch.einsum("hgd,nhd->hgn", q, key.double()).reshape(Hq, n) / 4
        s = torch.nn.functional.pad(s, (0, -n % 64), value=-math.inf).view(Hq, -1, 64).amax(-1)
        before = s.cummax(-1).values[:, :-1]
        grown = ((s[:, 1:] - before) > 8).sum(-1)
        assert bool((grown[odd[row]] >= 10).all())
        assert bool((s.amax(-1) - s[:, 0] < 8)[~odd[row]].any())
    for dtype in (F32, BF16):
        p.check(attend_paged(S, ws, p, scale=scale, out_dtype=dtype), True, scale=scale)
    assert S.device_status() == 0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def aliased(kv, Hq, Hkv, D, rows, pool=3, page=256):
    """A batch whose page tables name the same few pages over and over, so that long
    sequences need little memory: (pages and index arrays, queries)."""
    k, v = (randn(pool, Hkv, page, D, seed=s, dtype=BF16) for s in (kv[0] % 1000, 7))
    width = max(-(-n // page) for n in kv)
    table = torch.arange(width, device=DEV) % pool
    i32 = dict(dtype=torch.int32, device=DEV)
    where = (k, v, torch.arange(len(kv) + 1, **i32) * rows, torch.tensor(kv, **i32),
             table.to(torch.int32).expand(len(kv), -1).contiguous())
    return where, randn(rows * len(kv), Hq, D, seed=3, dtype=BF16)


def aliased_reference(where, q, n):
    """(out, size, spread) of one row on n such keys: each slot counts as often as a key
    lies in it."""
    pool, Hkv, page, D = where[0].shape
    i = torch.arange(pool * page, device=DEV)
    full, rest = divmod(n, pool * page)
    count = (full + (i < rest)).double()
    k, v = (x.transpose(1, 2).reshape(pool * page, Hkv, D).double() for x in where[:2])
    x = q[0].double().view(Hkv, -1, D)
    s = torch.einsum("hgd,nhd->hgn", x, k) * D ** -0.5
    p = torch.softmax(s + count.log(), -1)
    out = torch.einsum("hgn,nhd->hgd", p, v).reshape(1, -1, D)
    size = torch.einsum("hgn,nhd->hgd", p, v.abs()).reshape(1, -1, D)
    spread = (torch.einsum("hgd,nhd->hgn", x.abs(), k.abs()) * D ** -0.5).amax(-1)
    return out, size, spread.reshape(1, -1, 1)


@pytest.mark.parametrize("n, Hkv, D", [(4_100_003, 64, 64), (2_200_001, 128, 128),
                                       (300_000_001, 1, 64)], ids=str)
def test_long_lines_of_steps(S, ws, n, Hkv, D):
    """One sequence whose keys times kv heads are more than 2^28, with few rows."""
    where, q = aliased([n], Hkv, Hkv, D, 1)
    out = S.attention(q, *where, 1, ws, out_dtype=F32)
    assert S.device_status() == 0
    ref, size, spread = aliased_reference(where, q, n)
    # a warp adds to its sums once and to its outputs twice in each of its steps of 16 keys,
    # and the line is shared by 8 warps on each SM; parts are joined in under 200 additions
    steps = n * Hkv // 16 // (8 * sms()) + 200
    tol = attend_bound(ref, size, spread, 2 * 16 * steps, D, F32, False)
    assert bool(((out.double() - ref).abs() <= tol).all())
    assert float((tol / size).max()) < 0.02           # (so that a missing part would show)


def test_too_long_a_line_of_steps_is_recorded(S, ws):
    """2^27 steps of 32 kv heads: 2^32.  Nothing is written, and the workspace stays usable."""
    where, q = aliased([2 ** 31 - 512], 32, 32, 64, 1)
    out = torch.full_like(q, 5.0)
    S.attention(q, *where, 1, ws, out=out)
    assert S.device_status() == -5 and S.device_status() == 0
    assert bool((out == 5.0).all()) and not bool(ws[:4096].any())


@pytest.mark.parametrize("keys, rows", [
    (2 ** 31 - 512, 4200),     # 262 tiles of 2^24 units are more than 2^32
    (2 ** 26 + 2 ** 22, 4200)  # 262 tiles of 2^19 units and more: over 2^19 for each SM
], ids=str)
def test_too_long_a_line_of_units_is_recorded(S, ws, keys, rows):
    """Rows of 16 heads on one kv head, 256 a tile."""
    where, q = aliased([keys], 16, 1, 64, rows)
    out = torch.full_like(q, 5.0)
    S.attention(q, *where, rows, ws, out=out)
    assert S.device_status() == -5 and S.device_status() == 0
    assert bool((out == 5.0).all()) and not bool(ws[:4096].any())


def test_tiles_of_few_rows_of_long_sequences(S, ws):
    """A line of units that is long for its tiles, below the bound: one tile of 64 rows, each
    the same query, on 40M keys; the rows see all but the last few of them."""
    n, rows = 40_000_003, 16
    where, q = aliased([n], 4, 1, 64, rows)
    q[:] = q[:1]
    out = S.attention(q, *where, 64, ws, out_dtype=F32)
    assert S.device_status() == 0
    # a CTA's share: per 128 keys, 8 products are added to the outputs and two terms to the sum
    units = n // 128 // sms() + 200
    for r in (0, 7, rows - 1):
        ref, size, spread = aliased_reference(where, q, n - rows + r + 1)
        tol = attend_bound(ref, size, spread, 5 * 16 * units, 64, F32, True)
        assert bool(((out[r:r + 1].double() - ref).abs() <= tol).all())
        assert float((tol / size).max()) < 0.02


@pytest.mark.parametrize("joined", [False, True])
def test_append_to_a_part_of_a_batch(S, ws, joined):
    """Rows before row_start[0] belong to no sequence, like those from the last start on: the
    append and the attention both leave them alone, and nothing is recorded."""
    p = Paged([2, 3], [5, 8], 4, 2, 64, 16, DEV, joined=joined)
    n, T = 4, 4 + p.T + 60
    q, k, v = (randn(T, h, 64, seed=s, dtype=BF16) for h, s in ((4, 1), (2, 2), (2, 3)))
    starts = p.row_start + n
    k0, v0 = p.k_pages.clone(), p.v_pages.clone()
    out = torch.full_like(q, 3.0)
    S.kv_append(q, k, v, p.k_pages, p.v_pages, starts, p.kv_len, p.page_table, q_out=out)
    assert S.device_status() == 0
    assert torch.equal(out[n:n + p.T], q[n:n + p.T])
    assert bool((out[:n] == 3.0).all()) and bool((out[n + p.T:] == 3.0).all())
    for b, (r, length) in enumerate(zip(p.rows, p.kv)):
        i = torch.arange(length - r, length, device=DEV)
        pg, at = p.page_table[b, i // 16].long(), i % 16
        first = int(starts[b])
        assert torch.equal(p.k_pages[pg, :, at], k[first:first + r])
        k0[pg, :, at], v0[pg, :, at] = k[first:first + r], v[first:first + r]
    for old, new in ((k0, p.k_pages), (v0, p.v_pages)):
        assert torch.equal(old.view(torch.int16), new.view(torch.int16))
    got = torch.full_like(q, 3.0)
    S.attention(q, p.k_pages, p.v_pages, starts, p.kv_len, p.page_table, 3, ws, out=got)
    assert S.device_status() == 0
    p.check(got[n:n + p.T], True, q=q[n:n + p.T])
    assert bool((got[:n] == 3.0).all()) and bool((got[n + p.T:] == 3.0).all())


@pytest.mark.parametrize("starts", [[0, 5, 3], [0, 3, 2, 5, 6], [0, 2, 9], [-1, 2, 5], [0, -3, 5],
                                    [0] * 700 + [4, 3, 6]], ids=lambda s: str(s[-5:]))
@pytest.mark.parametrize("scale", [1, 66])
def test_append_records_row_starts_out_of_order(S, starts, scale):
    """Starts that are negative, fall or leave the rows are recorded, wherever they stand."""
    T, B = 6 * scale, len(starts) - 1
    p = Paged([1] * B, [400] * B, 4, 2, 64, 256, DEV)
    k = randn(T, 2, 64, dtype=BF16)
    good = [min(b * scale, T) for b in range(B + 1)]
    for s, status in ((good, 0), ([x * scale for x in starts], -5)):
        S.kv_append(None, k, k, p.k_pages, p.v_pages,
                    torch.tensor(s, dtype=torch.int32, device=DEV), p.kv_len, p.page_table)
        assert S.device_status() == status and S.device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("case", FEW, ids=str)
def test_few_rows_keep_p_in_fp32(S, ws, case, dtype):
    """The bound is for P as two bf16 halves; P rounded to bf16 is beyond it in each of these
    cases (test_attn_bounds)."""
    rows, kv, Hq, Hkv, D, page, window = case
    p = Paged(rows, kv, Hq, Hkv, D, page, DEV, seed=21)
    p.check(attend_paged(S, ws, p, window=window, out_dtype=dtype), False, window)
    assert S.device_status() == 0
