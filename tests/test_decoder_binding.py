"""What the Python binding of rope, kv_append and attention hands to the library:
no GPU, the tensors are on the host and the library is not called."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def S():
    from bit_expert_weight_gb300 import build
    build.build()
    import bit_expert_weight_gb300.smoe as S
    return S


@pytest.mark.parametrize("shape, strides", [
    ((5, 3, 64), (192, 64, 1)),      # contiguous
    ((5, 3, 64), (640, 64, 1)),      # a slice of one projection's output
    ((5, 3, 64), (64, 320, 1)),      # heads outermost
    ((5, 3, 64), (8, 64, 1)),        # rows of a sliding window: they overlap
    ((5, 3, 64), (64, 64, 1)),
    ((5, 1, 64), (8, 64, 1)),
    ((1, 3, 64), (8, 64, 1)),
    ((5, 3, 64), (0, 64, 1)),        # one row expanded
    ((5, 3, 64), (64, 0, 1)),        # one head expanded
    ((5, 3, 64), (1000, 72, 1)),
], ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_new_outputs_have_the_strides_that_are_passed(S, shape, strides, dtype):
    """The kernel writes by the strides it is given, the caller reads by the tensor's."""
    x = torch.as_strided(torch.zeros(8000), shape, strides)
    out, at, row, head = S._new_heads(x, dtype)
    assert out.shape == x.shape and out.dtype == dtype and out.data_ptr() == at
    assert out.is_contiguous() and (row, head) == (shape[1] * shape[2], shape[2])
    assert out.stride() == (row, head, 1)
