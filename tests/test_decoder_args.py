"""The rotation's frequency table, and what smoe_rope, smoe_kv_append and
smoe_attention refuse: host code, no GPU."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def S():
    from bit_expert_weight_gb300 import build
    build.build()
    import bit_expert_weight_gb300.smoe as S
    S.load()
    return S


def freqs(R, theta, kind="plain", factor=1.0, L0=4096.0, fast=32.0, slow=1.0):
    out = []
    for i in range(R // 2):
        f = theta ** (-2.0 * i / R)
        if kind == "linear":
            f /= factor
        elif kind == "parts":
            def at(turns):
                return R * math.log(L0 / (2 * math.pi * turns)) / (2 * math.log(theta))
            low, high = max(0, math.floor(at(fast))), min(R - 1, math.ceil(at(slow)))
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f * (1 - ramp) + f / factor * ramp
        elif kind == "bands":
            wave = 2 * math.pi / f
            if wave > L0 / slow:
                f /= factor
            elif wave >= L0 / fast:
                mix = (L0 / wave - slow) / (fast - slow)
                f = (1 - mix) * f / factor + mix * f
        out.append(f)
    return out


@pytest.mark.parametrize("kw", [
    dict(R=128, theta=1e6), dict(R=64, theta=1e4), dict(R=2, theta=1e4), dict(R=24, theta=5e5),
    dict(R=128, theta=1e4, kind="linear", factor=8.0),
    dict(R=128, theta=1e6, kind="parts", factor=16.0),
    dict(R=64, theta=1e4, kind="parts", factor=4.0, L0=32768.0, fast=16.0, slow=2.0),
    dict(R=128, theta=5e5, kind="bands", factor=8.0, L0=8192.0, fast=4.0, slow=1.0),
], ids=str)
def test_rope_table(S, kw):
    R, theta, kind = kw["R"], kw["theta"], kw.get("kind", "plain")
    table, scale = S.rope_table(R, theta, kind, kw.get("factor", 1.0), kw.get("L0", 4096.0),
                                kw.get("fast", 32.0), kw.get("slow", 1.0), device="cpu")
    ref = freqs(**kw)
    assert len(table) == R // 2
    for got, f in zip(table.tolist(), ref):
        want = f / (2 * math.pi)
        # double arithmetic on both sides: a few 2^-53, and one unit of the table
        assert abs(got * 2.0 ** -64 - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64
    want = 0.1 * math.log(kw["factor"]) + 1 if kind == "parts" else 1.0
    assert abs(scale - want) <= 2.0 ** -23 * want


def test_rope_table_refuses(S):
    L = S.load()
    out, sc = (ctypes.c_int64 * 128)(), ctypes.c_float()

    def call(R=128, theta=1e4, kind=0, factor=2.0, L0=4096.0, fast=32.0, slow=1.0, table=out):
        s = S.RopeScaling(kind, factor, L0, fast, slow)
        return L.smoe_rope_table(R, theta, ctypes.byref(s), table, ctypes.byref(sc))

    assert call() == 0
    for bad in (dict(R=0), dict(R=3), dict(R=258), dict(theta=1.0), dict(theta=math.inf),
                dict(theta=math.nan), dict(kind=4), dict(kind=-1), dict(kind=1, factor=0.5),
                dict(kind=1, factor=math.nan), dict(kind=2, L0=0.0), dict(kind=2, slow=0.0),
                dict(kind=3, fast=1.0), dict(kind=3, fast=math.inf), dict(table=None)):
        assert call(**bad) == -1, bad


PTR = 4096  # an aligned address that no refused call reads


def rope_args(S, **kw):
    d = dict(x=PTR, out=2 * PTR, x_row_stride=512, x_head_stride=128, out_row_stride=512,
             out_head_stride=128, num_rows=3, num_heads=4, head_dim=128, dtype=1, rot_dim=128,
             interleaved=0, rot_scale=1.0, eps=1e-6, positions=PTR, table=PTR, norm_w=None)
    d.update(kw)
    return S.RopeArgs(**d)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(out=None), dict(x=PTR + 8), dict(out=PTR + 2), dict(x_row_stride=516),
    dict(x_head_stride=-128), dict(out_head_stride=4), dict(num_rows=-1), dict(num_heads=-1),
    dict(num_heads=70000), dict(head_dim=0), dict(head_dim=100), dict(head_dim=264), dict(dtype=2),
    dict(rot_dim=0), dict(rot_dim=12), dict(rot_dim=136), dict(rot_scale=math.inf),
    dict(eps=-1.0), dict(eps=math.nan), dict(positions=None), dict(table=None),
    dict(table=PTR + 8), dict(norm_w=PTR + 8), dict(out=PTR, out_row_stride=1024),
], ids=str)
def test_rope_refuses(S, kw):
    assert S.load().smoe_rope(ctypes.byref(rope_args(S, **kw)), None) == -1


def test_nothing_to_do(S):
    L = S.load()
    assert L.smoe_rope(None, None) == -1
    assert L.smoe_rope(ctypes.byref(rope_args(S, num_rows=0, x=None)), None) == 0
    assert L.smoe_rope(ctypes.byref(rope_args(S, num_heads=0, x=None)), None) == 0
    assert L.smoe_kv_append(None, None) == -1
    assert L.smoe_kv_append(ctypes.byref(append_args(S, num_rows=0, k=None)), None) == 0
    assert L.smoe_kv_append(ctypes.byref(append_args(S, num_seqs=0, row_start=None)), None) == 0
    assert L.smoe_attention(None, None, 0, None) == -1
    for kw in (dict(num_rows=0, q=None), dict(num_seqs=0, row_start=None)):
        assert L.smoe_attention(ctypes.byref(attention_args(S, **kw)), None, 0, None) == 0


CACHE = dict(k_pages=PTR, v_pages=PTR, num_pages=10, k_page_stride=4 * 64 * 128,
             v_page_stride=4 * 64 * 128, page_size=64, num_kv_heads=4, head_dim=128,
             row_start=PTR, kv_len=PTR, page_table=PTR, num_rows=3, num_seqs=2, table_stride=5)

BAD_CACHE = [
    dict(k_pages=None), dict(v_pages=PTR + 2), dict(num_pages=0), dict(num_pages=1 << 31),
    dict(k_page_stride=4 * 64 * 128 - 8), dict(v_page_stride=4 * 64 * 128 + 4),
    dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(num_kv_heads=0),
    dict(head_dim=96), dict(head_dim=256), dict(row_start=None), dict(kv_len=None),
    dict(page_table=None), dict(num_rows=-1), dict(num_seqs=-1), dict(num_seqs=2049),
    dict(table_stride=-1),
]


def append_args(S, **kw):
    d = dict(CACHE, q=PTR, k=PTR, v=PTR, q_out=2 * PTR, q_row_stride=2048, q_head_stride=128,
             k_row_stride=512, k_head_stride=128, v_row_stride=512, v_head_stride=128,
             qo_row_stride=2048, qo_head_stride=128, num_heads=16, dtype=1, rot_dim=128,
             interleaved=0, rot_scale=1.0, eps=1e-6, positions=None, table=PTR, q_norm=None,
             k_norm=None)
    d.update(kw)
    return S.KvAppendArgs(**d)


@pytest.mark.parametrize("kw", BAD_CACHE + [
    dict(k=None), dict(v=None), dict(k=PTR + 8), dict(v_row_stride=4), dict(q=PTR + 4),
    dict(q_out=None), dict(num_heads=0), dict(num_heads=-1), dict(dtype=3), dict(rot_dim=136),
    dict(rot_dim=4), dict(table=None), dict(rot_scale=math.nan), dict(eps=-1.0),
    dict(rot_dim=0, eps=math.inf), dict(q_norm=PTR + 2), dict(k_norm=PTR + 8),
    dict(q_out=PTR, dtype=0), dict(q_out=PTR, qo_row_stride=4096),
], ids=str)
def test_append_refuses(S, kw):
    assert S.load().smoe_kv_append(ctypes.byref(append_args(S, **kw)), None) == -1


def attention_args(S, **kw):
    d = dict(CACHE, q=PTR, out=2 * PTR, q_row_stride=2048, q_head_stride=128, out_row_stride=2048,
             out_head_stride=128, num_heads=16, out_dtype=1, max_rows=2, window=0, scale=0.1)
    d.update(kw)
    return S.AttentionArgs(**d)


@pytest.mark.parametrize("kw", BAD_CACHE + [
    dict(q=None), dict(out=None), dict(q=PTR + 8), dict(out=PTR + 2), dict(out=PTR),
    dict(q_row_stride=2052), dict(out_head_stride=-8), dict(num_heads=0), dict(num_heads=18),
    dict(num_heads=4 * 129), dict(num_rows=1 << 28), dict(out_dtype=2), dict(max_rows=0), dict(window=-1),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
], ids=str)
def test_attention_refuses(S, kw):
    n = S.ATTENTION_WORKSPACE_BYTES
    assert S.load().smoe_attention(ctypes.byref(attention_args(S, **kw)), PTR, n, None) == -1


def test_attention_refuses_workspace(S):
    L, a, n = S.load(), attention_args(S), S.ATTENTION_WORKSPACE_BYTES
    assert L.smoe_attention(ctypes.byref(a), None, n, None) == -1
    assert L.smoe_attention(ctypes.byref(a), PTR + 128, n, None) == -1
    assert L.smoe_attention(ctypes.byref(a), PTR, n - 1, None) == -3


def test_binding_refuses(S):
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):   # not on the device
        S.rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        S.rope_table(64, 1e4, kind="other", device="cpu")
    with pytest.raises(S.SmoeError):
        S.rope_table(63, 1e4, device="cpu")
