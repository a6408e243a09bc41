"""The decoder layer over packed prompts without a GPU: what its workspace
holds, and what it checks of arguments that it does not read."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def D():
    from block_diffusion_speculative_step_gb300 import build
    build.build()
    import torch  # noqa: F401  (loads the shared CUDA runtime first, as in use)
    from block_diffusion_speculative_step_gb300 import dflash
    return dflash


H, NQ, NKV, HD, INTER = 4096, 32, 8, 128, 12288


def layer_args(D, M, dtype=None, norms=False, **kw):
    a = D.dflash_layer_args()
    a.dims = D.dflash_dims(H, NQ, NKV, HD, INTER, 151936, 1e6, 1e-6, D.DFLASH_BF16 if dtype is None else dtype)
    a.w = D.dflash_layer_weights(*[4096] * 6)
    a.n_seqs, a.rows, a.attn_mode = 3, M, D.DFLASH_ATTN_PROMPT
    a.h = a.rope_cs = a.tree_pos = a.prompt_start = 4096
    a.rope_max_pos = 1 << 20
    if norms:
        a.q_norm = a.k_norm = 4096
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("M", [2048, 8192, 65536])
def test_a_row_costs_its_own_activations(D, M, norms):
    """From a few launches' rows on, the workspace grows by what the rows
    themselves hold (norm, queries, keys, values, attention, activation in
    bf16; with head norms the projection in fp32), and by nothing for the
    projections' partial sums."""
    row = 2 * (H + 2 * NQ * HD + 2 * NKV * HD + INTER) + norms * 4 * (NQ + 2 * NKV) * HD
    a, b = (D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, layer_args(D, n, norms=norms)) for n in (M, 2 * M))
    assert 0 < b - a <= M * row + 4096  # (pieces are aligned to 256 bytes)


JUNK = [dict(pages=4104, page_size=100, max_pages=3, pool_pages=-1), dict(k=4104, v=8), dict(capacity=-5, window=7),
        dict(k_exp=4097, v_exp=3), dict(capacity=1 << 30)]


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("junk", JUNK)
def test_a_layer_without_a_context_takes_any_cache_descriptor(D, junk, norms):
    """base_pos NULL: kv is not read, nor checked.  (A workspace that is too
    small is the last thing that a call is refused for.)"""
    def call(**kw):
        a = layer_args(D, 100, norms=norms, **kw)
        for k, v in junk.items():
            setattr(a.kv, k, v)
        return a, D.lib().dflash_decoder_layer_forward(C.byref(a), C.c_void_p(256), 256, None)

    a, rc = call()
    assert rc == D.DFLASH_ERR_WORKSPACE, D.dflash_last_error()
    assert D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, a) == \
        D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, layer_args(D, 100, norms=norms))
    a, rc = call(base_pos=4096, max_pos=16)
    assert rc in (D.DFLASH_ERR_INVALID_ARG, D.DFLASH_ERR_UNSUPPORTED)


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("change,word", [(dict(k=4104), "aligned"), (dict(v=0), "NULL"), (dict(window=512), "window"),
                                         (dict(capacity=0), "capacity"), (dict(page_size=100, pages=4096), "page_size")])
def test_a_layer_over_a_context_checks_its_cache(D, change, word, norms):
    a = layer_args(D, 100, norms=norms, base_pos=4096, max_pos=512)
    a.kv = D.dflash_kv(4096, 4096, 512, 0)
    for k, v in change.items():
        setattr(a.kv, k, v)
    rc = D.lib().dflash_decoder_layer_forward(C.byref(a), C.c_void_p(256), 1 << 40, None)
    assert rc == D.DFLASH_ERR_INVALID_ARG and word in D.dflash_last_error(), D.dflash_last_error()
