"""The serving step that the README shows, run as it stands there."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from attn_helpers import attend, attend_bound  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def blocks():
    """The README's code of a step, and before it what is made once."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    part = text[text.index("Between the steps"):text.index("## Test")]
    code = re.findall(r"```python\n(.*?)```", part, re.S)
    return code[:-1], code[-1]


@pytest.mark.parametrize("page", [16, 32])
def test_readme_step(S, page):
    """Two requests of three beams: in every step the attention of both layers is that over the
    beams' own tokens, and the pool is closed up, so that nothing is lost where pages moved."""
    R, beams, D, H, Hkv, V, P, W = 2, 3, 64, 4, 2, 200, 90, 12
    g = torch.Generator(device=DEV).manual_seed(page)
    n, i32 = R * beams, dict(dtype=torch.int32, device=DEV)
    emb = torch.randn(V, H + 2 * Hkv, D, generator=g, device=DEV).bfloat16()
    head = 0.02 * torch.randn(H * D, V, generator=g, device=DEV).bfloat16()
    pages = torch.full((2, P, 2, Hkv, page, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    k_layers, v_layers = [p[:, 0] for p in pages], [p[:, 1] for p in pages]
    attn_ws, heard = S.attention_workspace(DEV), []

    def project(tokens):
        return emb[tokens.long()].split([H, Hkv, Hkv], dim=1)

    def model(tokens, row_start, kv_len, page_table):
        """Two layers that are alike, and a head on the last one."""
        q, k, v = project(tokens.view(-1))
        heard.clear()
        for kp, vp in zip(k_layers, v_layers):
            where = (kp, vp, row_start, kv_len, page_table)
            heard.append(S.attention(S.kv_append(q, k, v, *where), *where, 1, attn_ws))
        return heard[-1].flatten(1) @ head

    space = dict(
        S=S, torch=torch, model=model, beams=beams, page_size=page, k_layers=k_layers,
        v_layers=v_layers, refs=torch.zeros(P, **i32), kv_len=torch.zeros(n, **i32),
        page_table=torch.zeros(n, W, **i32), row_start=torch.arange(n + 1, **i32),
        scores=torch.zeros(R, beams, device=DEV),
        tokens=torch.randint(3, V, (R, beams), generator=g, **i32))
    once, step = blocks()
    for code in once:
        exec(code, space)
    refs, moved = space["refs"], 0
    refs[:5] = 1                              # held by the program itself, and then let go
    said = [[] for _ in range(n)]
    for turn in range(3 * page):
        if turn == page + 3:
            refs[:5] = 0
        said = [s + [t] for s, t in zip(said, space["tokens"].view(-1).tolist())]
        exec(step, space)
        moved += int(space["counts"][0])
        for s in range(n):
            q, k, v = project(torch.tensor(said[s], device=DEV))
            ref, size, wide = attend(q[-1:], k.double(), v.double(), 1, D ** -0.5, 0)
            tol = attend_bound(ref, size, wide, len(said[s]), D, torch.bfloat16, True)
            for a in heard:
                assert bool(((a[s:s + 1].double() - ref).abs() <= tol).all()), (turn, s)
        parents = space["parents"].view(-1).tolist()
        assert all(0 <= p < n for p in parents)
        said = [said[p] for p in parents]
        held = (refs > 0).nonzero()[:, 0].tolist()
        assert held == list(range(len(held)))
    assert moved > 0 and S.device_status() == 0
