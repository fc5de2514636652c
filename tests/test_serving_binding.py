"""Arrays whose sizes do not belong to one another, as the beams' and pages' calls of the
binding take them: host code, no GPU."""
import pytest

torch = pytest.importorskip("torch")

from test_pages_args import S, call, calls  # noqa: E402,F401 (fixtures)

I32 = torch.int32


@pytest.mark.parametrize("name", ["parent", "keep"])
@pytest.mark.parametrize("shape", [(2,), (4,), (6,), (2, 3), (0,)], ids=str)
def test_fork_takes_one_number_per_sequence(S, calls, name, shape):  # noqa: F811
    """Three sequences: more numbers than that (the parents of a selection of twice as many as
    there are beams) are of other sequences than those that they would be read for."""
    with pytest.raises(ValueError):
        call(S, "pages_fork", change={name: torch.zeros(shape, dtype=I32)})
    assert not calls.got


@pytest.mark.parametrize("shape", [(3,), (3, 1), (1, 3)], ids=str)
def test_fork_takes_any_shape_of_them(S, calls, shape):  # noqa: F811
    call(S, "pages_fork", change=dict(parent=torch.zeros(shape, dtype=I32),
                                      keep=torch.zeros(shape, dtype=I32)))
    call(S, "pages_fork", change=dict(keep=None))
    assert calls.got["smoe_pages_fork"][2] == 0
