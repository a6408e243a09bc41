"""Tree forwards at the end of a cache, lengths and positions outside their
bounds, and templates with rows that hold no node."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_tree_attn import PAD, TYPES, Tree, trees
from tests.test_gpu_tree_engine import engine, prompts_of, small, template

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("nq", [4, 64])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 257, 2 ** 31 - 1])
def test_length_outside_the_bound_is_reported(dtype, cache, nq, bad):
    p = Tree([200, 256, 90], trees(2, [5, 5, 4], 5), nq, 2, 128, dtype, cache, cap=300)
    p.a.max_pos = 256
    p.run()
    p.check()
    p.base[0] = bad
    p.run()
    p.check(D.DFLASH_ERR_INVALID_ARG, seqs=[1, 2])


@pytest.mark.parametrize("kv8", [False, True])
def test_tree_cycles_at_the_end_of_the_cache(kv8):
    """A tree's rows need no slots behind the context: cycles go on while the
    longest path fits, with every slot seen."""
    w = small("f32")
    prompts = prompts_of(w, 2, 100)
    n, N = 20, 65
    tree = template(5, N, w.block, 4)
    wide, eng = (engine(w, 3, 2, cap, tree=tree, kv8=kv8) for cap in (384, 128))
    for e in (wide, eng):
        e.prefill(prompts)
    done = 0
    while done < n:
        done += 1
        for e in (wide, eng):
            e.tree_cycle()
            assert e.status() == D.DFLASH_OK
        assert torch.equal(wide.h[:2 * N], eng.h[:2 * N])  # every row of the last layer's output
        assert torch.equal(wide.t_out, eng.t_out) and torch.equal(wide.base_pos, eng.base_pos)
        if int(eng.base_pos.max()) + w.block > 128:
            break
    assert int(eng.base_pos.max()) > 128 - N


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [-1, 134, 2 ** 31 - 1])
def test_position_outside_the_rope_table_is_reported(dtype, bad):
    """One node's position outside the table of cap + block positions; the
    same position in a padding row means nothing."""
    w = small(dtype)
    eng = engine(w, 3, 2, 128, tree=template(5, 9, w.block, 4))
    eng.prefill(prompts_of(w, 2))
    eng.tree_cycle()
    assert eng.status() == D.DFLASH_OK and eng.rope_max == 134
    keep = eng.t_pos.clone()
    for parent, want in ((None, D.DFLASH_ERR_INVALID_ARG), (PAD, D.DFLASH_OK)):
        eng.t_pos.copy_(keep)
        eng.t_pos[13] = bad
        if parent is not None:
            eng.t_parent[1, 4:] = parent
        a = eng.tree_layer_args(0, 9, eng.h, eng.t_pos, eng.t_parent)
        D.dflash_decoder_layer_forward(a, eng.ws_ptr, eng.ws_bytes)
        assert eng.status() == want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kv8", [False, True])
def test_template_with_rows_that_hold_no_node(dtype, kv8):
    """Padding rows (and rows below them) change nothing, whatever the
    workspace held before: the cycle's tokens are those of the tree without."""
    w = small(dtype)
    parent, rank = template(3, 12, w.block, 4)
    padded = parent + [PAD, PAD, 12], rank + [0, 0, 0]
    prompts = prompts_of(w, 2)
    got = []
    for tree in ((parent, rank), padded):
        eng = engine(w, 7, 2, tree=tree, kv8=kv8)
        eng.prefill(prompts)
        steps = []
        for _ in range(4):
            off = eng.ws_ptr - eng.ws.data_ptr() + 256 + (128 << 10)
            eng.ws[off:] = 0xFF  # NaN as bf16 and as fp32
            eng.tree_cycle()
            assert eng.status() == D.DFLASH_OK
            steps.append((eng.accept_len.cpu().tolist(), eng.t_out[:, :w.block].cpu().tolist(), eng.base_pos.cpu().tolist()))
        got.append(steps)
    if dtype == "f32":  # (bf16: the cut of the context goes by the launch)
        assert got[0] == got[1]


@pytest.mark.parametrize("dtype,cache", TYPES)
def test_bound_of_zero(dtype, cache):
    p = Tree([0, 0], trees(2, [5, 4], 5), 4, 2, 64, dtype, cache, cap=128)
    p.a.max_pos = 0
    p.run()
    p.check()


@pytest.mark.parametrize("kv8", [False, True])
def test_more_tree_rows_than_one_verification_takes(kv8):
    """9 sequences x 128 rows: several verification calls a cycle.  Every
    sequence gets what it gets alone."""
    w = small("f32")
    tree = template(4, 128, w.block, 4)
    prompts = prompts_of(w, 9)
    many = engine(w, 3, 9, tree=tree, kv8=kv8)
    out, acc = many.tree_generate(prompts, 6)
    assert many.status() == D.DFLASH_OK
    for s in (0, 7, 8):
        one = engine(w, 3, 1, tree=tree, kv8=kv8)
        o, a = one.tree_generate(prompts[s:s + 1], 6)
        assert one.status() == D.DFLASH_OK
        assert torch.equal(o[0], out[s]) and torch.equal(a[0], acc[s, :a.shape[1]])
