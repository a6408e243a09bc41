"""A packed layer of several thousand rows, whose projections run as many
launches over a few sets of partial sums."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_prompt_engine import engine, small

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[250] * 14 + [7], [256] * 5 + [100], [1200, 60, 1500], [255] * 20])
def test_many_launches_of_rows(lens):
    """bf16: every sequence's rows are as they are alone.  Keys and values are a
    projection of the rows themselves: the same bits.  The residuals differ by
    the attention's last bits (its work is cut by all the lengths), which may
    tip bf16 roundings of the two products behind it: 1e-2 as in a layer's
    other comparisons.  And the same bits every time."""
    w = small("bf16", H=512, nq=8, nkv=2, I=1408, t_layers=1, taps=(0, 0))
    eng = engine(w, 14, 1, 2048, norms=True)
    M, t = sum(lens), w.target
    g = torch.Generator(device="cuda").manual_seed(1)
    h0 = torch.randn(M, t.hidden, generator=g, device="cuda")
    eng._prompt_buffers(M, max(lens))
    a = eng.prompt_layer_args(0, len(lens), M, eng.ph, eng.ph, eng.ph)  # (the pointers do not matter here)
    assert D.dflash_workspace_bytes(D.DFLASH_OP_LAYER, a) <= eng.ws_bytes

    def run(h, ns):
        start = torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in ns]).cuda()
        h = h.clone()
        eng.pkb[0].zero_()
        eng.pvb[0].zero_()
        D.dflash_decoder_layer_forward(eng.prompt_layer_args(0, len(ns), sum(ns), h, start, pos), eng.ws_ptr, eng.ws_bytes)
        torch.cuda.synchronize()
        assert eng.status() == D.DFLASH_OK
        return h, eng.pkb[0][:sum(ns)].clone(), eng.pvb[0][:sum(ns)].clone()

    whole = run(h0, lens)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(whole, run(h0, lens)))
    r0 = 0
    for n in lens:
        h, k, v = run(h0[r0:r0 + n], [n])
        r = slice(r0, r0 + n)
        assert torch.equal(whole[1][r], k) and torch.equal(whole[2][r], v), r0
        assert float((whole[0][r] - h).abs().max()) < 1e-2, r0
        r0 += n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norms", [False, True])
def test_a_cache_descriptor_that_is_not_read(dtype, norms):
    """Without a context kv may hold anything."""
    w = small(dtype)
    eng = engine(w, 15, 2, norms=norms)
    M = 70
    eng._prompt_buffers(M, 40)
    start = torch.tensor([0, 30, M], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in (30, 40)]).cuda()
    h0 = torch.randn(M, w.target.hidden, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    out = []
    for junk in ({}, dict(k=8, v=0, pages=3, page_size=100, max_pages=-1, pool_pages=0, capacity=-7, window=5, k_exp=1)):
        h = h0.clone()
        a = eng.prompt_layer_args(0, 2, M, h, start, pos)
        for k, v in junk.items():
            setattr(a.kv, k, v)
        D.dflash_decoder_layer_forward(a, eng.ws_ptr, eng.ws_bytes)
        assert eng.status() == D.DFLASH_OK
        out.append(h)
    assert torch.equal(*out)
