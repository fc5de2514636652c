"""What the error bounds of the attention of few rows tell apart: P kept as two bf16 halves
passes the bound for it, P rounded to bf16 does not.  On the CPU, in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import Paged, gather  # noqa: E402

# rows and keys of each sequence; query heads, kv heads, head_dim, page, window: at most 32
# packed rows per sequence and kv head, of keys few enough that their rounding errors do not
# average out
FEW = [
    ([1], [7], 64, 4, 128, 16, 0),
    ([1], [300], 16, 1, 128, 64, 0),                       # one item in many parts
    ([1] * 8, [2, 15, 16, 17, 40, 64, 5, 130], 8, 8, 64, 16, 0),
    ([1, 1], [90, 250], 3, 1, 64, 128, 0),
    ([1] * 4, [100, 64, 65, 9000], 8, 2, 64, 16, 24),
    ([5] * 4, [5, 6, 130, 31], 24, 4, 128, 32, 0),
    ([7, 7, 0, 1], [7, 3, 60, 9000], 8, 2, 64, 64, 30),
    ([3], [200], 10, 1, 64, 16, 0),
    ([2, 32, 20], [40, 33, 21], 2, 2, 128, 16, 0),
]


def with_rounded_p(p, window, halves):
    """The attention in float64 but for P, held in one or two bf16 values."""
    out, at = [], 0
    for b, (r, n) in enumerate(zip(p.rows, p.kv)):
        if r == 0:
            continue
        k, v = (gather(x, p.page_table[b], n) for x in (p.k_pages, p.v_pages))
        q = p.q[at:at + r].double().view(r, p.Hkv, -1, p.D)
        s = torch.einsum("rhgd,nhd->hgrn", q, k) * p.D ** -0.5
        i = n - r + torch.arange(r)[:, None]
        j = torch.arange(n)[None, :]
        s = s.masked_fill((j > i) | (j <= i - (window or n + 1)), -math.inf)
        m = s.amax(-1, keepdim=True)
        e = (s - torch.where(m.isinf(), 0.0, m)).exp()
        held = e.bfloat16().double()
        if halves == 2:
            held = held + (e - held).bfloat16().double()
        l = e.sum(-1, keepdim=True)
        w = torch.where(l > 0, held / l, 0.0)
        out.append(torch.einsum("hgrn,nhd->rhgd", w, v).reshape(r, p.Hq, p.D))
        at += r
    return torch.cat(out).float()


@pytest.mark.parametrize("case", FEW, ids=str)
def test_bound_of_few_rows_tells_bf16_p_apart(case):
    rows, kv, Hq, Hkv, D, page, window = case
    assert max(rows) * Hq // Hkv <= 32
    p = Paged(rows, kv, Hq, Hkv, D, page, "cpu", seed=21)
    p.check(with_rounded_p(p, window, 2), False, window)
    one = with_rounded_p(p, window, 1)
    p.check(one, True, window)
    with pytest.raises(AssertionError):
        p.check(one, False, window)
