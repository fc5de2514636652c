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


class Placed:
    """A host tensor that says it lies on CUDA device `index`."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def __getitem__(self, at):
        return Placed(self.t[at], self.index)

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return self.index >= 0


class Handle:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


class Calls:
    """What reaches the library instead of it: name -> (packed arguments, the rest)."""

    def __init__(self):
        self.got = {}

    def __getattr__(self, name):
        def call(args, *rest):
            self.got[name] = (args, rest)
            return 0
        return call


@pytest.fixture
def calls(S, monkeypatch):
    lib = Calls()
    monkeypatch.setattr(S, "load", lambda: lib)
    monkeypatch.setattr(S, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 1000 + dev)
    return lib


def operands(S):
    """Arguments of the three calls by name; `where` says where each one lies."""
    i32, bf = torch.int32, torch.bfloat16
    pages = torch.zeros(4, 2, 16, 64, dtype=bf)
    batch = dict(k_pages=pages, v_pages=pages.clone(),
                 row_start=torch.zeros(2, dtype=i32), kv_len=torch.zeros(1, dtype=i32),
                 page_table=torch.zeros(1, 3, dtype=i32))
    x, kv = torch.zeros(5, 4, 64, dtype=bf), torch.zeros(5, 2, 64, dtype=bf)
    table, norm = torch.zeros(32, dtype=torch.int64), torch.zeros(64, dtype=bf)
    pos = torch.zeros(5, dtype=i32)
    ws = torch.empty(S.ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8)
    return {
        "rope": (S.rope, dict(x=x, positions=pos, table=table, norm_w=norm, out=x.clone())),
        "kv_append": (S.kv_append, dict(q=x, k=kv, v=kv.clone(), **batch, table=table, q_norm=norm,
                                        k_norm=norm.clone(), positions=pos, q_out=x.clone())),
        "attention": (S.attention, dict(q=x, **batch, ws=ws, out=x.clone())),
    }


def call(S, name, elsewhere=None, index=0, **kw):
    """The call with every tensor on device 0 but `elsewhere`, which is on device `index`."""
    f, args = operands(S)[name]
    args = {k: Placed(t, index if k == elsewhere else 0) for k, t in args.items()}
    if name == "attention":
        args["max_rows"] = 1
    args.update(kw)
    return f(**args)


NAMES = {
    "rope": ["x", "positions", "table", "norm_w", "out"],
    "kv_append": ["q", "k", "v", "k_pages", "v_pages", "row_start", "kv_len", "page_table", "table",
                  "q_norm", "k_norm", "positions", "q_out"],
    "attention": ["q", "k_pages", "v_pages", "row_start", "kv_len", "page_table", "ws", "out"],
}


@pytest.mark.parametrize("name", sorted(NAMES))
def test_calls_on_one_device_reach_the_library(S, calls, name):
    call(S, name)
    assert calls.got["smoe_" + name][1][-1] == 1000
    call(S, name, stream=Handle(0))
    assert calls.got["smoe_" + name][1][-1] == 77


@pytest.mark.parametrize("index", [-1, 1], ids=["host", "other device"])
@pytest.mark.parametrize("name, arg", [(n, a) for n in sorted(NAMES) for a in NAMES[n]])
def test_tensors_elsewhere_are_refused(S, calls, name, arg, index):
    """The kernel would read or write another device's, or the host's, addresses."""
    with pytest.raises(ValueError):
        call(S, name, arg, index)
    assert not calls.got


@pytest.mark.parametrize("name", sorted(NAMES))
def test_another_device_than_the_current_one_is_refused(S, calls, monkeypatch, name):
    """The library launches on the current device, with its status word."""
    with pytest.raises(ValueError):
        call(S, name, stream=Handle(1))
    monkeypatch.setattr(S, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        call(S, name)
    assert not calls.got


def test_workspaces_of_another_layout_are_refused(S, calls):
    n = S.ATTENTION_WORKSPACE_BYTES
    for ws in (torch.empty(1, dtype=torch.uint8).expand(n),
               torch.empty(2 * n, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            call(S, "attention", ws=Placed(ws, 0))
    assert not calls.got
    with pytest.raises(ValueError):
        S.attention_workspace("cpu")
    assert not calls.got


def unpacked(cls, raw):
    return cls.from_buffer_copy(raw)


def test_strides_of_dimensions_of_one_are_free(S, calls):
    """Nothing steps along a dimension of one, so its stride may be anything: one row out of
    a wider buffer, one kv head stored after its slots."""
    bf = torch.bfloat16
    one = torch.as_strided(torch.zeros(1000, dtype=bf), (1, 4, 64), (259, 64, 1))
    x = Placed(one, 0)
    pos, table = Placed(torch.zeros(1, dtype=torch.int32), 0), Placed(torch.zeros(32).long(), 0)
    S.rope(x, pos, table, out=x)
    a = unpacked(S.RopeArgs, calls.got["smoe_rope"][0])
    assert a.x_row_stride % 8 == 0 and a.out_row_stride == a.x_row_stride and a.x_head_stride == 64
    head = Placed(torch.as_strided(torch.zeros(1000, dtype=bf), (3, 1, 64), (64, 7, 1)), 0)
    S.rope(head, Placed(torch.zeros(3, dtype=torch.int32), 0), table, out=head)
    a = unpacked(S.RopeArgs, calls.got["smoe_rope"][0])
    assert a.x_head_stride % 8 == 0 and a.x_row_stride == 64
    # pages of one kv head, its dimension after the slots' or of an odd stride; one page
    pages = torch.zeros(4, 16, 1, 64, dtype=bf)
    for p, stride in ((pages.transpose(1, 2), 1024), (pages[:, :, 0].unsqueeze(1), 1024),
                      (torch.as_strided(pages, (4, 1, 16, 64), (1024, 5, 64, 1)), 1024),
                      (torch.as_strided(pages, (1, 1, 16, 64), (3, 5, 64, 1)), 1024)):
        call(S, "attention", k_pages=Placed(p, 0), v_pages=Placed(p, 0))
        a = unpacked(S.AttentionArgs, calls.got["smoe_attention"][0])
        assert (a.k_page_stride, a.v_page_stride) == (stride, stride) and a.num_kv_heads == 1
    calls.got.clear()
    wide = torch.zeros(4, 2, 32, 64, dtype=bf)
    for p in (wide[:, :, :16], wide[:, :, ::2], torch.zeros(4, 2, 16, 128, dtype=bf)[..., :64],
              torch.zeros(4, 16, 2, 64, dtype=bf).transpose(1, 2)):
        with pytest.raises(ValueError):
            call(S, "attention", k_pages=Placed(p, 0), v_pages=Placed(p, 0))
    assert not calls.got


def test_attention_refuses_more_rows_than_tiles_are_counted_for(S):
    """num_rows * num_heads is rounded up to whole tiles in 31 bits."""
    import ctypes
    from test_decoder_args import attention_args
    a = attention_args(S, num_rows=(1 << 27) - 31, num_heads=16)
    assert S.load().smoe_attention(ctypes.byref(a), 4096, S.ATTENTION_WORKSPACE_BYTES, None) == -1
