"""How far smoe_beam_select's normaliser is off: log(sum_u exp(x_u - max)), whose exponentials
and sums are in fp32, against 64 bits."""
import pytest

torch = pytest.importorskip("torch")

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


@pytest.mark.parametrize("dtype, rows, V", [(BF16, 2_048, 151_936), (F32, 512, 151_936),
                                            (F32, 512, 100_003), (BF16, 2_048, 1_000)], ids=str)
def test_normaliser(S, dtype, rows, V):
    """Each row's score is its normaliser rounded to fp32, so that the best value is what that
    rounding leaves (2^-20 at most of values up to 16), and its own rounding to fp32 is no more
    than 2^-44: what it is off by is the normaliser's error.  At most 2^-18, as smoe.h has it;
    the mean is printed."""
    g = torch.Generator(device=DEV).manual_seed(V)
    x = (2.0 * torch.randn(rows, V, generator=g, device=DEV)).to(dtype)
    norm = torch.empty(rows, dtype=torch.float64, device=DEV)
    for r in range(0, rows, 64):
        y = x[r:r + 64].double()
        norm[r:r + 64] = (y - y.amax(-1, keepdim=True)).exp().sum(-1).log()
    score = norm.float().view(-1, 1)
    got, parents, tokens = S.beam_select(x, score, 1, S.beam_workspace(DEV))
    assert S.device_status() == 0
    assert torch.equal(parents.view(-1), torch.arange(rows, device=DEV, dtype=torch.int32))
    assert torch.equal(x.gather(1, tokens.long()), x.amax(-1, keepdim=True))
    off = (got.double() - (score.double() - norm[:, None])).abs()
    print(f"normaliser of {rows} rows of {V} {dtype}: mean {float(off.mean()):.2e}, "
          f"largest {float(off.max()):.2e}")
    assert float(off.max()) <= 2.0 ** -18 + 2.0 ** -40
