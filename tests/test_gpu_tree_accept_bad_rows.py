"""dflash_tree_accept on rows that are no distribution: nothing is accepted
behind them, whatever their children."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_tree_accept import Accept

pytestmark = pytest.mark.gpu


def ends_at(p, s, k):
    """The walk of sequence s accepts k tokens, then a token of the vocabulary."""
    o = {n: t.cpu() for n, t in p.o.items()}
    assert int(o["accept_len"][s]) == k and int(o["commit_count"][s]) == k + 1
    path, toks = o["path"][s].tolist(), o["out_tokens"][s].tolist()
    assert all(x == -1 for x in path[k + 1:]) and all(x == -1 for x in toks[k + 1:])
    assert 0 <= toks[k] < p.V and int(o["next_anchor"][s]) == toks[k]
    assert int(p.dev["base_pos"][s]) == p.base[s] + k + 1


@pytest.mark.parametrize("bad", [np.nan, np.inf, "all -inf"])
@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("V", [40, 400, 20001])
@pytest.mark.parametrize("where", ["other", "child", "last child"])
def test_bad_target_row_ends_the_walk(bad, drawn, V, where):
    """The row of the root, and of the first node below it; every child would
    be accepted (u = 0)."""
    par = [-1, 0, 0, 0, 1, 1]
    p = Accept(3, 6, V, drawn=drawn, seed=10, parents=[par] * 3, u=0.0)
    for s, node, kids in ((0, 0, (1, 2, 3)), (1, 1, (4, 5))):
        toks = [int(p.tokens[s, i]) for i in kids]
        x = next(v for v in range(V) if v not in toks) if where == "other" else toks[0 if where == "child" else -1]
        if bad == "all -inf":
            p.target[s, node] = -np.inf
        else:
            p.target[s, node, x] = bad
    p.put()
    p.run()
    p.check(D.DFLASH_ERR_NUMERIC, seqs=[2])
    ends_at(p, 0, 0)
    ends_at(p, 1, 1)


@pytest.mark.parametrize("bad", [np.nan, np.inf, "all -inf"])
@pytest.mark.parametrize("where", ["other", "child"])
def test_bad_draft_row_ends_the_walk(bad, where):
    p = Accept(3, 5, 300, chain=True, seed=11, u=0.0, levels=5)
    for s, level in ((0, 0), (1, 1)):
        x = int(p.tokens[s, level + 1])
        if bad == "all -inf":
            p.draft[s, level] = -np.inf
        else:
            p.draft[s, level, x if where == "child" else (x + 1) % 300] = bad
    p.put()
    p.run()
    p.check(D.DFLASH_ERR_NUMERIC, seqs=[2])
    ends_at(p, 0, 0)
    ends_at(p, 1, 1)


def test_the_next_call_is_right():
    p = Accept(2, 6, 400, drawn=False, seed=12)
    keep = p.target.copy()
    p.target[0, 0, 7] = np.nan
    p.put()
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_ERR_NUMERIC
    p.target = keep
    p.put()
    p.run()
    p.check()
