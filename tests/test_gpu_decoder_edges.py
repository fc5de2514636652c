"""Edges of rope, kv_append and attention on the GPU: views whose rows overlap, row starts,
long lines of work, values and scores of large size."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import Paged, attend, attend_bound, turned, turned_bound  # noqa: E402
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
