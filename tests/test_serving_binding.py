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


@pytest.mark.parametrize("name", ["last", "out/0", "out/1", "out/2"])
def test_select_takes_rows_of_its_own_width(S, calls, name):  # noqa: F811
    """Two groups of three beams, four outputs: rows of another width would be read or written
    across one another; more rows than there are groups, or one long row, are not."""
    def with_shape(shape, dtype=I32):
        t = torch.zeros(shape, dtype=torch.float32 if name == "out/0" else dtype)
        if name == "last":
            return dict(last=t)
        out = [torch.zeros(2, 4), torch.zeros(2, 4, dtype=I32), torch.zeros(2, 4, dtype=I32)]
        out[int(name[-1])] = t
        return dict(out=out)

    wide = 3 if name == "last" else 4
    for shape in ((2, wide), (5, wide), (2 * wide,), (9 * wide,), (2, wide, 1)):
        call(S, "beam_select", change=with_shape(shape))
    calls.got.clear()
    for shape in ((2, wide + 1), (2, 2 * wide), (3, 2 * wide), (5, wide, 2)):
        with pytest.raises(ValueError):
            call(S, "beam_select", change=with_shape(shape))
    assert not calls.got


def test_compact_takes_a_table_of_its_own_width(S, calls):  # noqa: F811
    """Three sequences of seven entries: a table to write of other columns would get each row in
    another place; more rows, or one long row, are not."""
    for shape in ((3, 7), (5, 7), (21,), (40,)):
        call(S, "pages_compact", change=dict(page_table_out=torch.zeros(shape, dtype=I32)))
    calls.got.clear()
    for shape in ((3, 8), (3, 14), (4, 6), (2, 20)):
        with pytest.raises(ValueError):
            call(S, "pages_compact", change=dict(page_table_out=torch.zeros(shape, dtype=I32)))
    assert not calls.got


@pytest.mark.parametrize("name", ["pages_fork", "pages_reserve", "pages_compact"])
def test_tables_of_one_dimension_are_refused(S, calls, name):  # noqa: F811
    with pytest.raises(ValueError):
        call(S, name, change=dict(page_table=torch.zeros(21, dtype=I32)))
    assert not calls.got
