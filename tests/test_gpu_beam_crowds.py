"""smoe_beam_select where very many logits are the largest finite number, or above it, with
NaNs among them, against its 64-bit definition."""
import math

import pytest

torch = pytest.importorskip("torch")

from pages_helpers import check_selection  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
LARGEST = torch.finfo(F32).max


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


def crowd(rows, V, dtype, largest):
    """Rows of `largest` in different places, a NaN before each of its runs."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.randn(rows, V, generator=g, device=DEV)
    i = torch.arange(V, device=DEV)
    for r in range(rows):
        kind = r % 5
        if kind == 0:                         # all but the first token
            x[r] = largest
            x[r, 0] = math.nan
        elif kind == 1:                       # all but every third
            x[r] = torch.where(i % 3 == 0, math.nan, largest)
        elif kind == 2:                       # a half, so that most of the row lies below
            x[r, :V // 2] = largest
            x[r, :V // 2:7] = math.nan
        elif kind == 3:                       # the other half, behind NaNs
            x[r, :V // 2] = math.nan
            x[r, V // 2:] = largest
        else:                                 # one of them, and NaNs
            x[r] = math.nan
            x[r, V - 3] = largest
    return x.to(dtype)


@pytest.mark.parametrize("largest", [math.inf, LARGEST, -math.inf], ids=["inf", "max", "none"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("rows, V", [(5, 5_000), (320, 5_000), (10, 70_001), (5, 1_023)],
                         ids=str)
def test_nan_among_the_largest(S, rows, V, dtype, largest):
    """A NaN is never chosen: not where the row's largest logits fill more than the kernel's
    queue, in one part of a row (320 rows) and in several."""
    x, ws = crowd(rows, V, dtype, largest), S.beam_workspace(DEV)
    # (+inf counts as the largest finite fp32, so the definition is given that)
    counted = x.float().clamp(max=LARGEST)
    for K in (1, 5):
        scores = -torch.arange(rows, device=DEV).float().view(-1, K)
        for n in (1, 4, 32):
            out = S.beam_select(x, scores, n, ws)
            assert S.device_status() == 0
            chosen = out[1].flatten().long(), out[2].flatten().long()
            found = chosen[0] >= 0
            assert not bool(x[chosen[0][found], chosen[1][found]].isnan().any())
            check_selection(out, counted, scores, n)
