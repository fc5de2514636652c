"""What smoe_pages_compact says of lengths in tables without columns."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
I32 = torch.int32


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


@pytest.mark.parametrize("P", [20, 140_003])   # by one launch, by four
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("lens", [(0, 5, 0), (-1, 0, 0), (0, 0, 2 ** 31 - 1), (0, 0, 0), (7,)],
                         ids=str)
def test_compact_records_lengths_without_columns(S, P, apart, lens):
    """A row of no columns has room for no keys: any other length is recorded, as in tables
    with columns; the pool is closed up all the same."""
    refs = torch.zeros(P, dtype=I32, device=DEV)
    refs[[1, 4, P - 1]] = torch.tensor([1, 2, 3], dtype=I32, device=DEV)
    kv = torch.tensor(lens, dtype=I32, device=DEV)
    table = torch.zeros(len(lens), 0, dtype=I32, device=DEV)
    out = dict(refs_out=torch.full((P,), 9, dtype=I32, device=DEV),
               page_table_out=table.clone()) if apart else {}
    copies = torch.full((P // 2, 2), -5, dtype=I32, device=DEV)
    counts = torch.zeros(2, dtype=I32, device=DEV)
    S.pages_compact(refs, kv, table, 16, copies, counts, **out)
    assert S.device_status() == (-5 if any(lens) else 0) and S.device_status() == 0
    assert counts.tolist() == [2, 3] and copies[:3].tolist() == [[4, 0], [P - 1, 2], [-5, -5]]
    now = out.get("refs_out", refs)
    assert now[:3].tolist() == [2, 1, 3] and not bool(now[3:].any())
    assert kv.tolist() == list(lens)
