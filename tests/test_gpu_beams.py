"""smoe_beam_select on the GPU against its 64-bit definition."""
import math

import pytest

torch = pytest.importorskip("torch")

from pages_helpers import check_selection  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


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


@pytest.fixture(scope="module")
def ws(S):
    return S.beam_workspace(DEV)


def rand(*shape, seed=0, spread=2.0, dtype=F32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (spread * torch.randn(*shape, generator=g, device=DEV)).to(dtype)


def select(S, ws, x, scores, n, **kw):
    out = S.beam_select(x, scores, n, ws, **kw)
    assert S.device_status() == 0
    assert not bool(ws[:8192].any())          # the counters are as they were
    check_selection(out, x, scores, n, kw.get("last"), kw.get("end_token", -1))
    return out


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("G, K, V, N", [
    (1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 7, 32), (1, 4, 8, 4), (3, 2, 31, 2), (1, 32, 100, 32),
    (5, 4, 1_001, 8), (2, 5, 4_099, 10), (1, 4, 32_000, 4), (7, 1, 8_192, 1), (2, 16, 8_193, 32),
    (1, 2, 300_007, 32), (40, 8, 3_000, 16), (2048, 1, 40, 3), (64, 32, 9, 32),
    (1, 1, 3_000_001, 5),
], ids=str)
def test_select(S, ws, G, K, V, N, dtype):
    x = rand(G * K, V, seed=G + V, dtype=dtype)
    select(S, ws, x, rand(G, K, seed=1), N)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("offset, stride", [(0, 1_003), (1, 1_003), (3, 1_000), (5, 1_024),
                                            (7, 4_000), (2, 0), (1, 1), (6, 999)], ids=str)
def test_rows_anywhere(S, ws, offset, stride, dtype):
    """Rows that begin at any multiple of the type, lie apart, overlap or are one."""
    buf = rand(40_000, seed=3, dtype=dtype)
    x = torch.as_strided(buf, (6, 997), (stride, 1), offset)
    a = select(S, ws, x, rand(2, 3, seed=4), 6)
    if stride % 8 == 0:                      # (all rows are aligned alike)
        b = S.beam_select(x.contiguous() if stride else x.clone(), rand(2, 3, seed=4), 6, ws)
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("V", [5, 64, 1_000, 70_001])
def test_ties_go_to_the_lowest(S, ws, V, dtype):
    """All logits alike, all scores alike: sums are whole numbers, so every value is the
    same; the first tokens of the first beams win.  -0 is equal to 0."""
    x = torch.zeros(8, V, dtype=dtype, device=DEV)
    x[:, ::2] = -0.0
    scores = torch.full((2, 4), -1.5, device=DEV)
    s, p, t = S.beam_select(x, scores, 12, ws)
    want = torch.arange(12, device=DEV)
    for g in range(2):
        assert p[g].tolist() == (4 * g + want // V).tolist() and t[g].tolist() == (want % V).tolist()
    tol = 2.0 ** -24 * (1.5 + math.log(V)) + 1e-12
    assert bool(((s.double() + 1.5 + math.log(V)).abs() <= tol).all())
    x[:, V // 2:] = 1.0                      # two sizes of logits
    select(S, ws, x, scores, 12)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_rising_and_falling_logits(S, ws, dtype):
    """Every element a new maximum, or none: the lists' slow path all the time, or once."""
    up = torch.linspace(-30, 40, 30_011, device=DEV)
    x = torch.stack([up, up.flip(0), -up, up * 3]).to(dtype)
    select(S, ws, x, torch.zeros(1, 4, device=DEV), 32)
    far = torch.stack([up * 1e4, up.flip(0) * 1e4]).to(dtype)
    select(S, ws, far, torch.zeros(2, 1, device=DEV), 7)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_masked_logits(S, ws, dtype):
    """-inf, NaN, the type's lowest and largest values, +inf; rows that are all of one."""
    low, inf, nan = torch.finfo(dtype).min, math.inf, math.nan
    x = rand(16, 5_003, seed=8, dtype=dtype)
    x[0] = -inf
    x[1] = nan
    x[2] = low
    x[3] = -inf
    x[3, 4_321] = 2.0
    x[4, 10:] = low
    x[5, ::3] = nan
    x[6, 1::2] = -inf
    x[7, [7, 70, 700]] = torch.finfo(dtype).max
    x[8, 1:] = -inf
    x[8, 0] = low
    x[9, 77] = torch.finfo(dtype).max
    x[9, 78] = low
    x[10, [8, 4_999]] = inf                  # as the largest finite fp32
    x[11, 5] = inf
    x[11, 6:] = low
    for K in (1, 2, 4, 16):
        for n in (1, 6, 32):
            select(S, ws, x, rand(16 // K, K, seed=K, spread=1.0), n)


def test_beams_without_continuations(S, ws):
    """Scores of -inf, +inf and NaN, finished beams, groups with fewer continuations than
    asked for; a beam that is not read may hold anything."""
    inf, nan = math.inf, math.nan
    scores = torch.tensor([[0.0, -inf, -inf, -inf], [-inf] * 4, [-1.0, -2.0, nan, inf],
                           [-3.0, -1.0, -2.0, -inf], [-5.0, -4.0, -inf, -6.0]], device=DEV)
    last = torch.full((5, 4), 9, dtype=I32, device=DEV)
    last[3, 0] = last[3, 1] = last[4, 1] = last[0, 1] = 2
    for V in (3, 11, 5_000):
        x = rand(20, V, seed=V)
        x[5] = nan
        x[12:14] = nan
        for n in (1, 4, 8, 32):
            select(S, ws, x, scores, n, last=last, end_token=2)
            select(S, ws, x, scores, n)                           # no end token, no last
            select(S, ws, x, scores, n, last=last)                # end_token -1
    last[:] = 2
    s, p, t = select(S, ws, x, scores, 4, last=last, end_token=2)
    assert t[2].tolist() == [2, 2, -1, -1] and p[2].tolist() == [8, 9, -1, -1]
    assert s[2, :2].tolist() == [-1.0, -2.0]


def test_large_scores_and_logits_keep_64_bits(S, ws):
    """Values are compared in 64 bits: logits that differ by 2^-10 under scores of -1e6, where
    fp32 sums could not tell them apart."""
    V = 2_000
    x = (torch.arange(V, device=DEV).float() * 2.0 ** -10).repeat(3, 1)
    x[1] = x[1].flip(0)
    scores = torch.tensor([[-1e6, -1e6, -1e6 - 0.5]], device=DEV)
    select(S, ws, x, scores, 16)


def test_in_place_repeated_and_captured(S, ws):
    """A captured step that works in place, replayed on other logits, equals calls by
    themselves; the same inputs give the same bits; a workspace serves all shapes."""
    G, K, V = 3, 4, 9_001
    xs = [rand(G * K, V, seed=s, dtype=BF16) for s in range(4)]
    x, scores = xs[0].clone(), torch.zeros(G, K, device=DEV)
    last = torch.full((G, K), 7, dtype=I32, device=DEV)
    parents = torch.zeros(G, K, dtype=I32, device=DEV)
    want, sc, la = [], scores.clone(), last.clone()
    for y in xs:
        for _ in range(2):
            again = S.beam_select(y, sc, K, ws, last=la, end_token=2)
        check_selection(again, y, sc, K, la, 2)
        other = S.beam_select(xs[0][:5], torch.zeros(5, 1, device=DEV), 3, ws)  # another shape
        assert torch.equal(other[2], S.beam_select(xs[0][:5], torch.zeros(5, 1, device=DEV), 3,
                                                   ws)[2])
        sc, _, la = again
        want.append(again)
    stream = torch.cuda.Stream()
    own = S.beam_workspace(DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        S.beam_select(x, scores, K, own, last=last, end_token=2, out=(scores, parents, last))
    for y, (s, p, t) in zip(xs, want):
        x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(scores, s) and torch.equal(parents, p) and torch.equal(last, t)
    assert S.device_status() == 0


def test_two_streams_at_once(S):
    """Two calls that overlap, each with a workspace, on streams of their own."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [S.beam_workspace(DEV) for _ in range(2)]
    xs = [rand(64, 40_000, seed=s, dtype=BF16) for s in (1, 2)]
    sc = [rand(8, 8, seed=s) for s in (3, 4)]
    want = [S.beam_select(x, s, 8, spaces[0]) for x, s in zip(xs, sc)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(S.beam_select(xs[i], sc[i], 8, spaces[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_few_of_the_vocabulary_allowed(S, ws, dtype):
    """Fewer tokens allowed than asked for, the rest at the type's lowest value: the lowest
    tokens of those make up the number."""
    x = torch.full((8, 60_001), torch.finfo(dtype).min, dtype=dtype, device=DEV)
    for r in range(8):
        x[r, torch.randperm(60_001, device=DEV)[:r]] = rand(r, seed=r, dtype=dtype)
    for K, n in ((1, 32), (2, 20), (8, 32)):
        select(S, ws, x, rand(8 // K, K, seed=1), n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
@pytest.mark.parametrize("spread", [0.0, 1e-2, 30.0])
def test_large_logits_close_together(S, ws, dtype, spread):
    """The large logits all lie where one warp reads them, or a few hundred words hold nothing
    else; many are alike in bf16, all where spread is 0."""
    V = 90_000
    i = torch.arange(V, device=DEV)
    per = 4 if dtype == F32 else 8
    near = rand(4, V, seed=3, spread=max(spread, 1e-9))
    x = torch.where((i // per) % 256 < 32, 100.0, 0.0) + near
    x[1] = torch.where(i < 3_000, 50.0, 0.0) + near[1]
    x[2] = torch.where(i > V - 3_000, 50.0, 0.0) + near[2]
    x[3] = torch.where((i // per) % 256 == 7, 50.0, 0.0) + near[3]
    if spread == 0:
        x = x.round()
    for K in (1, 4):
        for n in (2, 32):
            select(S, ws, x.to(dtype), rand(4 // K, K, seed=K), n)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_largest_vocabulary(S, ws, dtype):
    """2^22 tokens, the best ones at both ends and alike."""
    V = 1 << 22
    x = rand(2, V, seed=6, dtype=dtype)
    x[0, [0, V // 2, V - 1]] = 30.0
    x[1, [V - 2, V - 1]] = 30.0
    for K in (1, 2):
        s, p, t = select(S, ws, x, torch.zeros(2 // K, K, device=DEV), 5)
        if K == 1:
            assert t[0, :3].tolist() == [0, V // 2, V - 1] and t[1, :2].tolist() == [V - 2, V - 1]


def test_rows_far_apart(S, ws):
    """Rows whose offsets pass 32 bits."""
    buf = torch.empty(2 ** 32 + 20_000, dtype=BF16, device=DEV)
    x = torch.as_strided(buf, (3, 9_001), (2 ** 31 + 1, 1), 5)
    x.copy_(rand(3, 9_001, seed=2, dtype=BF16))
    a = S.beam_select(x, rand(1, 3, seed=3), 8, ws)
    assert S.device_status() == 0
    check_selection(a, x.clone(), rand(1, 3, seed=3), 8)


def test_end_token_without_last_tokens(S, ws):
    x = rand(6, 500, seed=1)
    a = select(S, ws, x, rand(2, 3, seed=2), 3, end_token=2)
    b = S.beam_select(x, rand(2, 3, seed=2), 3, ws)
    assert all(torch.equal(y, z) for y, z in zip(a, b))


def test_first_call_in_a_capture(S):
    """A process whose first calls are made while a graph is captured."""
    import subprocess
    import sys
    code = """
import torch, bit_expert_weight_gb300.smoe as S
d = dict(dtype=torch.int32, device="cuda:0")
ws, aws = torch.zeros(S.BEAM_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda:0"), None
x, sc = torch.randn(4, 5000, device="cuda:0"), torch.zeros(2, 2, device="cuda:0")
out = (torch.zeros(2, 2, device="cuda:0"), torch.zeros(2, 2, **d), torch.zeros(2, 2, **d))
refs, kv, table = torch.zeros(64, **d), torch.zeros(4, **d), torch.zeros(4, 8, **d)
start, copies, counts = torch.arange(5, **d) * 20, torch.zeros(32, 2, **d), torch.zeros(2, **d)
k, v = torch.zeros(64, 1, 16, 64, dtype=torch.bfloat16, device="cuda:0"), None
v = k.clone()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    S.beam_select(x, sc, 2, ws, out=out)
    S.pages_fork(refs, kv, table, 16, out[1].view(-1))
    S.pages_reserve(refs, kv, table, 16, start, copies, counts)
    S.pages_copy(k, v, copies[:4], counts)
    S.pages_compact(refs, kv, table, 16, copies, counts)
g.replay()
torch.cuda.synchronize()
assert kv.tolist() == [20] * 4 and counts.tolist() == [0, 8], (kv, counts)
assert out[1].tolist()[0][0] in (0, 1) and S.device_status() == 0
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
