"""Workspaces that an engine replaced."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_prompt_engine import engine, prompts_of, small

pytestmark = pytest.mark.gpu


def kept(eng):
    return sum(t.numel() for t, _ in eng.old_ws)


@pytest.mark.parametrize("kind", ["trees", "prompts"])
def test_what_is_kept_takes_no_more_than_the_last(kind):
    """Needs that grow a little at a time."""
    w = small("bf16")
    eng = engine(w, 16, 4, 1024)
    first = eng.ws_bytes
    for n in range(8, 129, 8):
        if kind == "trees":
            eng.set_tree([-1] + list(range(n - 1)), [0] * n)
        else:
            eng.prefill(prompts_of(w, [n * 7, 5, 1, n]))
    assert eng.ws_bytes > first and len(eng.old_ws) >= 1  # (or the case is none)
    assert kept(eng) <= eng.ws.numel()
    assert eng.status() == D.DFLASH_OK


def test_a_cycle_captured_before_a_larger_tree():
    """The graph of a chain cycle goes on in the workspace that it was captured with."""
    w = small("bf16")
    eng, ref = engine(w, 17, 2, 1024), engine(w, 17, 2, 1024)
    for e in (eng, ref):
        e.prefill(prompts_of(w, [9, 4]))
        e.cycle()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eng.cycle()
    before = eng.ws_ptr
    eng._new_workspace(eng.ws_bytes + 1)
    assert eng.ws_ptr != before
    for _ in range(4):
        g.replay()
        ref.cycle()
        assert torch.equal(eng.out_tokens, ref.out_tokens) and torch.equal(eng.base_pos, ref.base_pos)
    assert eng.status() == D.DFLASH_OK and ref.status() == D.DFLASH_OK
