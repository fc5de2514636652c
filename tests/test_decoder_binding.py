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


OVERLAPPING = [  # rows, heads, row stride, head stride of an output of heads of 128
    (3, 4, 0, 128), (3, 4, 120, 128), (3, 4, 512, 0), (3, 4, 512, 64), (2, 1, 64, 128),
    (1, 2, 512, 120),
]


@pytest.mark.parametrize("rows, heads, row, head", OVERLAPPING, ids=str)
def test_outputs_that_overlap_themselves_are_refused(S, rows, heads, row, head):
    """Two rows or two heads of one output in the same place: which one stays is left to
    chance, so the library refuses (as the inputs do not, which are only read)."""
    import ctypes
    from test_decoder_args import append_args, attention_args, rope_args
    L = S.load()
    out = dict(out_row_stride=row, out_head_stride=head, num_rows=rows)
    assert L.smoe_rope(ctypes.byref(rope_args(S, num_heads=heads, **out)), None) == -1
    a = attention_args(S, num_heads=heads, num_kv_heads=1, **out)
    assert L.smoe_attention(ctypes.byref(a), 4096, S.ATTENTION_WORKSPACE_BYTES, None) == -1
    a = append_args(S, num_heads=heads, num_rows=rows, qo_row_stride=row, qo_head_stride=head)
    assert L.smoe_kv_append(ctypes.byref(a), None) == -1
