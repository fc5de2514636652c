"""What the beams' and pages' calls refuse, in the library and in the binding, and the plain
definitions themselves: host code, no GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from pages_helpers import Pool, check_selection, random_pool, values  # noqa: E402
from test_decoder_binding import Calls, Handle, Placed  # noqa: E402

PTR = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def S():
    from bit_expert_weight_gb300 import build
    build.build()
    import bit_expert_weight_gb300.smoe as S
    S.load()
    return S


def beam_args(S, **kw):
    d = dict(logits=PTR, row_stride=100, scores=2 * PTR, last=3 * PTR, scores_out=4 * PTR,
             parents=5 * PTR, tokens=6 * PTR, dtype=1, vocab=100, num_groups=2, beams=4, num_out=8,
             end_token=2)
    d.update(kw)
    return S.BeamArgs(**d)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=PTR + 1), dict(logits=PTR + 2, dtype=0), dict(row_stride=-1),
    dict(row_stride=(1 << 40) + 1), dict(scores=None), dict(scores_out=None), dict(parents=None),
    dict(tokens=None), dict(dtype=2), dict(vocab=0), dict(vocab=(1 << 22) + 1),
    dict(num_groups=-1), dict(num_groups=513), dict(beams=0), dict(beams=33), dict(num_out=0),
    dict(num_out=33), dict(end_token=-2), dict(end_token=100), dict(scores_out=2 * PTR),
    dict(tokens=3 * PTR), dict(parents=6 * PTR), dict(parents=3 * PTR, num_out=4),
], ids=str)
def test_select_refuses(S, kw):
    n = S.BEAM_WORKSPACE_BYTES
    assert S.load().smoe_beam_select(ctypes.byref(beam_args(S, **kw)), PTR, n, None) == -1


def test_select_refuses_workspace(S):
    L, a, n = S.load(), beam_args(S), S.BEAM_WORKSPACE_BYTES
    assert L.smoe_beam_select(ctypes.byref(a), None, n, None) == -1
    assert L.smoe_beam_select(ctypes.byref(a), PTR + 128, n, None) == -1
    assert L.smoe_beam_select(ctypes.byref(a), PTR, n - 1, None) == -3


def pool_args(S, **kw):
    d = dict(refs=PTR, kv_len=2 * PTR, page_table=3 * PTR, num_pages=1000, page_size=16,
             num_seqs=8, table_stride=40)
    d.update(kw)
    return S.PagePool(**d)


BAD_POOL = [dict(refs=None), dict(refs=PTR + 8), dict(kv_len=None), dict(page_table=None),
            dict(num_pages=0), dict(num_pages=(1 << 30) + 1), dict(page_size=8),
            dict(page_size=48), dict(page_size=512), dict(page_size=0), dict(num_seqs=-1),
            dict(num_seqs=2049), dict(table_stride=-1), dict(table_stride=(1 << 27) + 1)]


@pytest.mark.parametrize("kw", BAD_POOL, ids=str)
def test_pools_are_refused(S, kw):
    L, p = S.load(), ctypes.byref(pool_args(S, **kw))
    assert L.smoe_pages_fork(p, 5 * PTR, None, None) == -1
    assert L.smoe_pages_reserve(p, 5 * PTR, 6 * PTR, 7 * PTR, None) == -1
    assert L.smoe_pages_compact(p, 5 * PTR, 6 * PTR, 7 * PTR, 1 << 30, 8 * PTR, None) == -1


def test_fork_and_reserve_refuse(S):
    L, p = S.load(), ctypes.byref(pool_args(S))
    assert L.smoe_pages_fork(None, 5 * PTR, None, None) == -1
    assert L.smoe_pages_fork(p, None, None, None) == -1
    assert L.smoe_pages_fork(p, 2 * PTR, None, None) == -1          # the lengths themselves
    assert L.smoe_pages_fork(p, 5 * PTR, 2 * PTR, None) == -1
    assert L.smoe_pages_reserve(None, 5 * PTR, 6 * PTR, 7 * PTR, None) == -1
    for bad in ((None, 6 * PTR, 7 * PTR), (5 * PTR, None, 7 * PTR), (5 * PTR, 6 * PTR, None)):
        assert L.smoe_pages_reserve(p, *bad, None) == -1
    empty = ctypes.byref(pool_args(S, num_seqs=0, kv_len=None, page_table=None))
    assert L.smoe_pages_fork(empty, None, None, None) == 0


def test_compact_refuses(S):
    L, p = S.load(), ctypes.byref(pool_args(S))
    far = 100 * PTR
    for bad in ((None, far, far, 500, far), (far, None, far, 500, far), (far, far, None, 500, far),
                (far, far, far, 499, far), (far, far, far, 500, None), (far, far, far + 4, 500, far),
                (PTR + 16, far, far, 500, far), (PTR - 400, far, far, 500, far),
                (PTR + 3984, far, far, 500, far), (far, 3 * PTR + 64, far, 500, far),
                (far, 3 * PTR - 64, far, 500, far)):
        assert L.smoe_pages_compact(p, *bad, None) == -1, bad
    assert L.smoe_pages_compact(None, far, far, far, 500, far, None) == -1


CACHE = dict(k_pages=PTR, v_pages=2 * PTR, num_pages=10, k_page_stride=4 * 64 * 128,
             v_page_stride=4 * 64 * 128, page_size=64, num_kv_heads=4, head_dim=128)


def copy_call(S, changes, num_caches=None, copies=PTR, counts=PTR, most=5):
    caches = (S.KvCache * len(changes))(*[S.KvCache(**dict(CACHE, **c)) for c in changes])
    n = len(changes) if num_caches is None else num_caches
    return S.load().smoe_pages_copy(caches, n, copies, counts, most, None)


@pytest.mark.parametrize("kw", [
    dict(k_pages=None), dict(v_pages=PTR + 2), dict(num_pages=0), dict(k_page_stride=64),
    dict(v_page_stride=4 * 64 * 128 + 4), dict(page_size=48), dict(num_kv_heads=0),
    dict(head_dim=96),
], ids=str)
def test_copy_refuses_caches(S, kw):
    assert copy_call(S, [kw]) == -1
    assert copy_call(S, [{}, kw]) == -1


@pytest.mark.parametrize("kw", [
    dict(num_pages=11), dict(k_page_stride=8 * 64 * 128), dict(v_page_stride=8 * 64 * 128),
    dict(page_size=32), dict(num_kv_heads=2), dict(head_dim=64)], ids=str)
def test_copy_refuses_caches_of_different_sizes(S, kw):
    assert copy_call(S, [kw, {}]) == -1


def test_copy_refuses(S):
    assert copy_call(S, [{}], num_caches=-1) == -1
    assert copy_call(S, [{}], num_caches=129) == -1
    assert copy_call(S, [{}], copies=None) == -1
    assert copy_call(S, [{}], counts=None) == -1
    assert copy_call(S, [{}], most=-1) == -1
    assert S.load().smoe_pages_copy(None, 1, PTR, PTR, 5, None) == -1
    assert S.load().smoe_pages_copy(None, 0, None, None, 5, None) == 0
    assert copy_call(S, [{}], most=0) == 0


def test_nothing_to_select(S):
    L = S.load()
    assert L.smoe_beam_select(None, PTR, S.BEAM_WORKSPACE_BYTES, None) == -1
    assert L.smoe_beam_select(ctypes.byref(beam_args(S, num_groups=0, logits=None)), None, 0,
                              None) == 0


# --------------------------------------------------------------- the binding

@pytest.fixture
def calls(S, monkeypatch):
    class Any(Calls):
        def __getattr__(self, name):
            def call(*args):
                self.got[name] = args
                return 0
            return call
    lib = Any()
    monkeypatch.setattr(S, "load", lambda: lib)
    monkeypatch.setattr(S, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(S, "_raw_stream", lambda dev: 1000 + dev)
    return lib


def operands(S):
    i32, bf = torch.int32, torch.bfloat16
    pool = dict(refs=torch.zeros(20, dtype=i32), kv_len=torch.zeros(3, dtype=i32),
                page_table=torch.zeros(3, 7, dtype=i32))
    pages = torch.zeros(4, 2, 16, 64, dtype=bf)
    pairs, counts = torch.zeros(10, 2, dtype=i32), torch.zeros(2, dtype=i32)
    three = torch.zeros(3, dtype=i32)
    return {
        "beam_select": (S.beam_select, dict(
            logits=torch.zeros(6, 50, dtype=bf), scores=torch.zeros(2, 3),
            last=torch.zeros(2, 3, dtype=i32), out=[torch.zeros(2, 4), torch.zeros(2, 4, dtype=i32),
                                                    torch.zeros(2, 4, dtype=i32)],
            ws=torch.empty(S.BEAM_WORKSPACE_BYTES, dtype=torch.uint8)),
            dict(num_out=4, end_token=2)),
        "pages_fork": (S.pages_fork, dict(**pool, parent=three, keep=three.clone()),
                       dict(page_size=16)),
        "pages_reserve": (S.pages_reserve, dict(**pool, row_start=torch.zeros(4, dtype=i32),
                                                copies=pairs, counts=counts), dict(page_size=16)),
        "pages_copy": (S.pages_copy, dict(k_pages=[pages, pages], v_pages=[pages, pages],
                                          copies=pairs, counts=counts), {}),
        "pages_compact": (S.pages_compact, dict(**pool, copies=pairs, counts=counts,
                                                refs_out=pool["refs"].clone(),
                                                page_table_out=pool["page_table"].clone()),
                          dict(page_size=16)),
    }


NAMES = ["beam_select", "pages_fork", "pages_reserve", "pages_copy", "pages_compact"]
TENSORS = [(n, a, i) for n, args in (
    ("beam_select", ["logits", "scores", "last", "ws", "out/0", "out/1", "out/2"]),
    ("pages_fork", ["refs", "kv_len", "page_table", "parent", "keep"]),
    ("pages_reserve", ["refs", "kv_len", "page_table", "row_start", "copies", "counts"]),
    ("pages_copy", ["k_pages/0", "v_pages/1", "copies", "counts"]),
    ("pages_compact", ["refs", "kv_len", "page_table", "copies", "counts", "refs_out",
                       "page_table_out"])) for a in args for i in (-1, 1)]


def call(S, name, elsewhere=None, index=0, change=None, **kw):
    """The call with every tensor on device 0 but `elsewhere`, which is on device `index`."""
    f, args, rest = operands(S)[name]
    placed = {}
    for k, t in dict(args, **(change or {})).items():
        if isinstance(t, list):
            placed[k] = [Placed(x, index if elsewhere == f"{k}/{i}" else 0)
                         for i, x in enumerate(t)]
        else:
            placed[k] = None if t is None else Placed(t, index if k == elsewhere else 0)
    return f(**placed, **dict(rest, **kw))


@pytest.mark.parametrize("name", NAMES)
def test_calls_reach_the_library(S, calls, name):
    call(S, name)
    assert calls.got["smoe_" + name][-1] == 1000
    call(S, name, stream=Handle(0))
    assert calls.got["smoe_" + name][-1] == 77


@pytest.mark.parametrize("name, arg, index", TENSORS)
def test_tensors_elsewhere_are_refused(S, calls, name, arg, index):
    with pytest.raises(ValueError):
        call(S, name, arg, index)
    assert not calls.got


@pytest.mark.parametrize("name", NAMES)
def test_another_device_than_the_current_one_is_refused(S, calls, monkeypatch, name):
    with pytest.raises(ValueError):
        call(S, name, stream=Handle(1))
    monkeypatch.setattr(S, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError):
        call(S, name)
    assert not calls.got


@pytest.mark.parametrize("name, change, error", [
    ("beam_select", dict(logits=torch.zeros(6, 50, dtype=torch.float16)), TypeError),
    ("beam_select", dict(logits=torch.zeros(5, 50)), ValueError),
    ("beam_select", dict(logits=torch.zeros(50, 6).T), ValueError),
    ("beam_select", dict(scores=torch.zeros(2, 3, dtype=torch.float64)), ValueError),
    ("beam_select", dict(last=torch.zeros(5, dtype=torch.int32)), ValueError),
    ("beam_select", dict(ws=torch.empty(64 << 20, dtype=torch.uint8)[::2]), ValueError),
    ("pages_fork", dict(parent=torch.zeros(3, dtype=torch.int64)), ValueError),
    ("pages_fork", dict(parent=torch.zeros(2, dtype=torch.int32)), ValueError),
    ("pages_fork", dict(page_table=torch.zeros(2, 7, dtype=torch.int32)), ValueError),
    ("pages_fork", dict(page_table=torch.zeros(3, 14, dtype=torch.int32)[:, ::2]), ValueError),
    ("pages_reserve", dict(row_start=torch.zeros(3, dtype=torch.int32)), ValueError),
    ("pages_reserve", dict(copies=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    ("pages_reserve", dict(counts=torch.zeros(1, dtype=torch.int32)), ValueError),
    ("pages_copy", dict(v_pages=[torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)]), ValueError),
    ("pages_copy", dict(copies=torch.zeros(20, dtype=torch.int32)), ValueError),
    ("pages_compact", dict(copies=torch.zeros(20, dtype=torch.int32)), ValueError),
    ("pages_compact", dict(refs_out=torch.zeros(19, dtype=torch.int32)), ValueError),
    ("pages_compact", dict(page_table_out=torch.zeros(20, dtype=torch.int32)), ValueError),
], ids=lambda x: str(x)[:40] if not isinstance(x, dict) else ",".join(x))
def test_binding_refuses(S, calls, name, change, error):
    with pytest.raises(error):
        call(S, name, change=change)
    assert not calls.got


def test_row_strides_are_handed_on(S, calls):
    wide = torch.zeros(6, 80, dtype=torch.bfloat16)
    for x, stride in ((wide[:, :50], 80), (wide[:1].expand(6, 80), 0),
                      (torch.as_strided(wide, (6, 50), (3, 1)), 3)):
        call(S, "beam_select", change=dict(logits=x))
        a = S.BeamArgs.from_buffer_copy(calls.got["smoe_beam_select"][0])
        assert (a.row_stride, a.vocab, a.num_groups, a.beams) == (stride, x.shape[1], 2, 3)


# --------------------------------------------------------------- the definitions

def test_pool_definition():
    """By hand: two sequences of 20 keys on pages of 16, the second a copy of the first."""
    p = Pool(6, 16, 3, 4)
    assert p.reserve([20, 0, 0]) == ([], 4) and p.table[0][:2] == [0, 1]
    p.fork([0, 0, -1])
    assert p.refs == [2, 2, 0, 0, 0, 0] and p.kv == [20, 20, 0]
    assert p.reserve([1, 1, 3]) == ([[1, 2]], 2)
    assert p.table[0][:2] == [0, 1] and p.table[1][:2] == [0, 2] and p.table[2][:1] == [3]
    assert p.refs == [2, 1, 1, 1, 0, 0]
    assert p.reserve([48, 0, 0]) is None and p.kv == [21, 21, 3]
    p.fork([-1, 1, 2], [9, 9, 40])
    assert p.refs == [1, 0, 0, 1, 0, 0] and p.kv == [0, 9, 3]
    assert p.compact() == ([[3, 1]], 2) and p.table[2][0] == 1 and p.refs == [1, 1, 0, 0, 0, 0]


def test_random_pools_are_sound():
    for seed in range(20):
        p = random_pool(60, 16, 9, 12, seed)
        count = [0] * 60
        for s in range(9):
            for q in p.used(s):
                count[q] += 1
        assert count == p.refs


def test_check_selection_tells_wrong_answers_apart():
    """The right answer passes; a wrong token, order, score or a missed one does not."""
    g = torch.Generator().manual_seed(0)
    x, sc = torch.randn(6, 40, generator=g), torch.randn(2, 3, generator=g)
    v = values(x, sc).flatten(1)
    s, at = v.sort(descending=True, stable=True)
    good = [s[:, :5].float(), (at[:, :5] // 40 + torch.tensor([[0], [3]])).int(),
            (at[:, :5] % 40).int()]
    check_selection(good, x, sc, 5)
    for i, change in ((0, lambda t: t + 1e-3), (2, lambda t: (t + 1) % 40),
                      (2, lambda t: t.flip(1)), (1, lambda t: t.roll(1, 0)),
                      (0, lambda t: t.flip(1))):
        bad = list(good)
        bad[i] = change(good[i])
        with pytest.raises(AssertionError):
            check_selection(bad, x, sc, 5)
    later = [s[:, 1:6].float(), (at[:, 1:6] // 40 + torch.tensor([[0], [3]])).int(),
             (at[:, 1:6] % 40).int()]
    with pytest.raises(AssertionError):
        check_selection(later, x, sc, 5)
