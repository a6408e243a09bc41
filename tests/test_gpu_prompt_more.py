"""Packed prompts through the engine: other shapes, paged rings, an engine that
is used again, another stream."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests import gpu_common as G
from tests.test_gpu_prompt_engine import Engine, engine, model, prompts_of, small, target64

pytestmark = pytest.mark.gpu


def near(u, v):
    return float((u - v).abs().max()) < 1e-5 * max(1.0, float(u.abs().max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [dict(H=384, nq=6, nkv=2, d=128, I=640), dict(H=256, nq=8, nkv=1, d=128, I=384),
                                   dict(H=256, nq=3, nkv=3, d=64, I=264)])
@pytest.mark.parametrize("piece", [0, 50])
def test_scores_of_other_shapes(dtype, shape, piece):
    """As test_scores, at its tolerances; no alternatives asked for."""
    w = small(dtype, **shape)
    prompts = prompts_of(w, [1, 140, 33])
    m = model(w, 30, True)
    eng = Engine(w, G.to_dev(m), 3, 256)
    tol = 1e-4 if dtype == "f32" else 2 * G.LOGIT_TOL["bf16"]
    for p, (lp, ent, ids, top) in zip(prompts, eng.score(prompts, piece=piece)):
        ref = torch.log_softmax(target64(w, m, p), -1)
        n = p.numel()
        assert ids.shape == top.shape == (n, 0) and lp.shape == (n - 1,)
        if n > 1:
            want = ref[:-1].gather(1, p.cpu().long()[1:, None])[:, 0]
            assert float((lp.cpu().double() - want).abs().max()) < tol
        assert float((ent.cpu().double() + (ref.exp() * ref).sum(-1)).abs().max()) < tol
    assert eng.status() == D.DFLASH_OK


@pytest.mark.parametrize("piece", [0, 70])
def test_paged_window_rings(piece):
    """Draft rings in pages, with prompts longer and shorter than the window."""
    w = small("f32", window=128)
    prompts = prompts_of(w, [200, 40, 300])
    a, b = engine(w, 31, 3, 512), engine(w, 31, 3, 512)
    b.page_caches(128, seed=5, spare_pages=3)
    a.prefill(prompts)
    b.prefill_packed(prompts, piece)
    for _ in range(3):
        a.cycle()
        b.cycle()
        assert torch.equal(a.out_tokens, b.out_tokens) and torch.equal(a.base_pos, b.base_pos)
    x, y = (e.unpaged_caches()["d"] for e in (a, b))
    for s, n in enumerate(a.base_pos.tolist()):
        for u, v in zip(x[0] + x[1], y[0] + y[1]):
            assert near(u[s, :, :min(n, 128)], v[s, :, :min(n, 128)])
    assert a.status() == D.DFLASH_OK and b.status() == D.DFLASH_OK


def test_an_engine_used_again():
    """Shorter prompts after longer ones, packed after uniform ones: as on a new engine."""
    w = small("f32")
    first, then = prompts_of(w, [180, 150]), prompts_of(w, [20, 3])
    used, new = engine(w, 32, 2, norms=True), engine(w, 32, 2, norms=True)
    used.score(first, topk=2)
    used.prefill(torch.stack([p[:100] for p in first]))
    for _ in range(3):
        used.cycle()
    for e in (used, new):
        e.prefill(then)
    for _ in range(4):
        used.cycle()
        new.cycle()
        assert torch.equal(used.out_tokens, new.out_tokens) and torch.equal(used.base_pos, new.base_pos)
    assert used.status() == D.DFLASH_OK and new.status() == D.DFLASH_OK


def test_on_another_stream():
    w = small("bf16")
    prompts = prompts_of(w, [90, 7, 31])
    a, b = engine(w, 33, 3), engine(w, 33, 3)
    x = a.score(prompts, topk=3)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = b.score(prompts, topk=3)
    st.synchronize()
    assert torch.equal(a.anchor, b.anchor)
    for u, v in zip(x, y):
        assert all(torch.equal(i, j) for i, j in zip(u, v))
    assert a.status() == D.DFLASH_OK and b.status() == D.DFLASH_OK
