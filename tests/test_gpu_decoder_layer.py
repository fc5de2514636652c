"""The operators together, as a serving loop uses them: a decoder layer over a paged
cache, prompts in chunks beside single tokens, against the same rows in one piece and
against a plain computation of the attention half."""
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import UBF, attend, turned  # noqa: E402
from test_decoder_args import freqs  # noqa: E402

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
    import decoder_layer
    decoder_layer.S.load()
    decoder_layer.S.device_status()
    return decoder_layer


@pytest.fixture(scope="module")
def layer(ex):
    return ex.DecoderLayer(ex.Y.WORKLOADS["tiny"], 8, 2, 64, torch.device(DEV))


def rows_of(layer, lens):
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    return [torch.randn(n, layer.wl.d, generator=g, device=DEV).bfloat16() for n in lens]


def attention_half(ex, layer, cache, xs, pieces):
    """The attention's output of every row, the rows of each sequence fed in `pieces`
    (a list of row counts per step and sequence)."""
    done, out = [0] * len(xs), [[] for _ in xs]
    for rows in pieces:
        batch = cache.grow(rows)
        x = torch.cat([x[d:d + r] for x, d, r in zip(xs, done, rows)])
        q, k, v = layer.project(x)
        where = (cache.k_pages, cache.v_pages, *batch)
        q = ex.S.kv_append(q, k, v, *where, layer.rope, layer.rot_scale, q_norm=layer.q_norm,
                           k_norm=layer.k_norm, eps=ex.EPS)
        a = ex.S.attention(q, *where, max(rows), layer.attn_ws, out_dtype=torch.float32)
        at = 0
        for b, r in enumerate(rows):
            out[b].append(a[at:at + r])
            at += r
            done[b] += r
    assert ex.S.device_status() == 0
    return [torch.cat(o) for o in out]


@pytest.mark.parametrize("pieces", [
    [[150, 33, 1]],
    [[64, 33, 1], [64, 0, 0], [22, 0, 0]],
    [[100, 30, 0], [1, 1, 0], [1, 1, 1], [47, 1, 0], [1, 0, 0]],
    [[4, 1, 1]] * 8 + [[3, 1, 0]] * 25 + [[43, 0, 0]],
], ids=["whole", "chunks", "mixed", "drafts"])
def test_attention_half_in_pieces(ex, layer, pieces):
    lens = [sum(p[b] for p in pieces) for b in range(3)]
    xs = rows_of(layer, lens)
    cache = ex.PagedCache(40, 16, 2, 64, 3, 16, torch.device(DEV))
    got = attention_half(ex, layer, cache, xs, pieces)
    freq = torch.tensor(freqs(64, 1e6, "parts", 4.0), dtype=torch.float64, device=DEV)
    for x, out in zip(xs, got):
        n = x.shape[0]
        if n == 0:
            continue
        # the keys and values as the cache rounds them; the products of the
        # pieces may differ in their last bit from the whole's, by one rounding
        # of q, k and v to bf16 each
        pos = torch.arange(n, device=DEV)
        q, k, v = layer.project(x)
        q, _ = turned(q, pos, freq, layer.rot_scale, False, layer.q_norm, ex.EPS)
        k, _ = turned(k, pos, freq, layer.rot_scale, False, layer.k_norm, ex.EPS)
        q, k = q.to(torch.bfloat16), k.to(torch.bfloat16)
        ref, size, spread = attend(q, k.double(), v.double(), n, 64 ** -0.5, 0)
        # each score is off by two roundings of its two factors (projection and
        # rotation: 4 x 2^-8 of sum |q||k|), p twice that (in p and in the sum);
        # v by one, p itself by one
        tol = size * (2 * 4 * UBF * spread + 2 * UBF) + 1e-6
        err = (out.double() - ref).abs()
        assert bool((err <= tol).all()), f"worst {float((err / tol).max())} of the bound"


def test_layer_runs_and_pages_are_reused(ex, layer):
    """The whole layer in chunks equals the whole layer in one piece, up to bf16 roundings of
    its output; a sequence that takes over another's pages sees none of its keys."""
    xs = rows_of(layer, [90])
    dev = torch.device(DEV)
    one = ex.PagedCache(8, 16, 2, 64, 1, 8, dev)
    ref = layer(xs[0], one, one.grow([90]), 90).double()
    cache = ex.PagedCache(8, 16, 2, 64, 1, 8, dev)
    cache.k_pages.fill_(math.nan)
    cache.v_pages.fill_(math.nan)
    for turn in range(2):
        parts = []
        for a, b in ((0, 40), (40, 41), (41, 90)):
            parts.append(layer(xs[0][a:b], cache, cache.grow([b - a]), b - a))
        got = torch.cat(parts).double()
        off = (got - ref).abs().max() / ref.abs().max()
        assert float(off) <= 8 * UBF, (turn, float(off))
        cache.drop(0)
        cache.free.reverse()
    assert ex.S.device_status() == 0


def test_example_runs(ex):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py")],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "done: [5, 5, 5, 5] tokens made" in r.stdout
