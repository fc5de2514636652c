"""The beams' and pages' operators together with the append and the attention, as a search
uses them: every beam's attention is that over its own tokens, whatever its pages went
through; and the example."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import attend, attend_bound  # noqa: E402
from pages_helpers import Pool, check_selection  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_expert_weight_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import beam_search
    beam_search.S.load()
    beam_search.S.device_status()
    return beam_search


@pytest.mark.parametrize("beams, page, lens, spread", [
    (4, 16, [37, 5, 64], 1.0), (1, 32, [20, 1], 1.0), (5, 16, [16, 15, 17, 1], 0.02),
    (8, 64, [130], 0.05),
], ids=str)
def test_beams_attend_to_their_own_tokens(ex, beams, page, lens, spread):
    S, R, D, V = ex.S, len(lens), 64, 300
    model = ex.TinyModel(V, 4, 2, D, torch.device(DEV), seed=beams)
    model.head *= spread                      # flat logits: the beams mix more
    search = ex.BeamSearch(model, R, beams, 400, page, 16, D, 2, torch.device(DEV))
    search.k_pages.fill_(float("nan"))        # nothing that was not written is used
    search.v_pages.fill_(float("nan"))
    g = torch.Generator().manual_seed(page)
    prompts = [torch.randint(3, V, (n,), generator=g).tolist() for n in lens]
    said = [list(p) if k == 0 else [] for p in prompts for k in range(beams)]
    plain = Pool(400, page, R * beams, 16, fill=0)
    seen = {}

    def watch(tokens, row_start, max_rows, attend_=search.attend):
        a = attend_(tokens, row_start, max_rows)
        seen.update(rows=row_start.diff().tolist(), a=a)
        want = plain.reserve(seen["rows"])
        assert search.counts.tolist() == [len(want[0]), want[1]]
        return a

    def chosen(logits, choose=search.choose):
        before = search.scores.clone(), search.tokens.clone()
        choose(logits)
        check_selection((search.scores, search.parents, search.tokens), logits, before[0], beams,
                        before[1], 2)
        plain.fork(search.parents.view(-1).tolist())

    search.attend, search.choose = watch, chosen
    for step in range(14):
        if step == 0:
            search.prompts(prompts)
        else:
            search.step()
        at = 0
        for s, r in enumerate(seen["rows"]):
            if r == 0:
                continue
            q, k, v = model.project(torch.tensor(said[s], device=DEV))
            ref, size, wide = attend(q[-r:], k.double(), v.double(), r, D ** -0.5, 0)
            tol = attend_bound(ref, size, wide, len(said[s]), D, torch.bfloat16, True)
            assert bool(((seen["a"][at:at + r].double() - ref).abs() <= tol).all()), (step, s)
            at += r
        parents, tokens = search.parents.view(-1).tolist(), search.tokens.view(-1).tolist()
        said = [said[p] + [max(t, 0)] if p >= 0 else [max(t, 0)] for p, t in zip(parents, tokens)]
        assert search.kv_len.tolist() == plain.kv and search.refs.tolist() == plain.refs
        assert search.table.tolist() == plain.table
        assert [len(x) - 1 for x in said] == plain.kv
    assert S.device_status() == 0


def test_example_runs(ex):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "beam_search.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "done:" in r.stdout and r.stdout.count("request") == 3


def test_a_captured_step(ex):
    """The whole step of a search (room, copies, append, attention, choice, reordering) as one
    graph, replayed: what it comes to is the same as call by call, to the bit."""
    def begin():
        model = ex.TinyModel(300, 4, 2, 64, torch.device(DEV), seed=9)
        search = ex.BeamSearch(model, 3, 4, 300, 16, 16, 64, 2, torch.device(DEV))
        search.prompts([[5] * 40, list(range(3, 20)), [7]])
        return search

    eager, replayed = begin(), begin()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    eager.step()                              # (libraries are ready before the capture)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        replayed.step()
    for step in range(40):
        if step:
            eager.step()
        graph.replay()
        for a, b in ((eager.parents, replayed.parents), (eager.tokens, replayed.tokens),
                     (eager.refs, replayed.refs), (eager.kv_len, replayed.kv_len),
                     (eager.table, replayed.table), (eager.counts, replayed.counts),
                     (eager.scores, replayed.scores)):
            assert torch.equal(a, b), step
    assert ex.S.device_status() == 0
