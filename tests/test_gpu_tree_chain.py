"""A chain as a tree: the chain cycle and the tree cycle over the chain of the
draft's tokens are the same computation, over either cache."""
import numpy as np
import pytest

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_tree_engine import engine, prompts_of, small

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("S", [1, 3])
def test_chain_cycles_are_tree_cycles(kv8, S):
    w = small("f32", 0)
    prompts = prompts_of(w, S)
    B = w.block
    chain = engine(w, 3, S, kv8=kv8)
    tree = engine(w, 3, S, tree=(list(range(-1, B - 1)), [0] * B), kv8=kv8)
    a, ka = chain.speculative_generate(prompts, 24)
    b, kb = tree.tree_generate(prompts, 24)
    assert chain.status() == D.DFLASH_OK and tree.status() == D.DFLASH_OK
    np.testing.assert_array_equal(a.numpy(), b.numpy())
    np.testing.assert_array_equal(ka.numpy(), kb.numpy())
