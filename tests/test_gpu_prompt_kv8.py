"""Packed prompts committed to an 8-bit cache: every slot's codes and exponents."""
import numpy as np
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.test_gpu_prompt_engine import engine, prompts_of, small
from tests.tree_ref import quantise_row

pytestmark = pytest.mark.gpu

LENS = [40, 9, 130]


def caches(eng):
    c = eng.caches
    return list(zip(c.tk + c.tv, c.tke + c.tve)) if eng.kv8 else c.tk + c.tv


def values(codes, ex):
    return codes.view(torch.float8_e4m3fn).double() * torch.exp2(ex.double() - 127)[..., None]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norms", [False, True])
def test_codes_are_those_of_the_unquantised_rows(dtype, norms):
    """A prompt's rows see each other unquantised, so the same pass over a cache
    of the network's type holds the rows that the 8-bit one quantises: equal
    codes and exponents at every position, and nothing behind them."""
    w = small(dtype)
    a, b = engine(w, 12, 3, norms=norms, kv8=True), engine(w, 12, 3, norms=norms)
    for e in (a, b):
        e.prefill(prompts_of(w, LENS))
        assert e.status() == D.DFLASH_OK
    for (codes, ex), rows in zip(caches(a), caches(b)):
        codes, ex, rows = codes.cpu().numpy(), ex.cpu().numpy(), rows.double().cpu().numpy()
        for s, n in enumerate(LENS):
            for g in range(w.target.n_kv):
                for p in range(n):
                    c, e = quantise_row(rows[s, g, p])
                    assert e == ex[s, g, p] and np.array_equal(c, codes[s, g, p]), (s, g, p)
            assert not codes[s, :, n:].any() and not ex[s, :, n:].any(), s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_sequence_s_cache_is_as_alone(dtype):
    """Each sequence's slots against the same prompt alone.  The first layer's rows
    are projections of the tokens: the same codes.  Later ones differ by the
    attention's last bits and the roundings that these tip: 1e-5 (fp32) or 2e-2
    (bf16) of the row's size, and on either side half a step of e4m3, 2^-4 of the
    value or 2^-10 of the scale.  By the same bound no sequence passes for another."""
    w = small(dtype)
    prompts = prompts_of(w, LENS)
    eng = engine(w, 12, 3, norms=True, kv8=True)
    eng.prefill(prompts)
    alone = []
    for p in prompts:
        one = engine(w, 12, 1, norms=True, kv8=True)
        one.prefill([p])
        assert one.status() == D.DFLASH_OK and one.base_pos[0] == p.numel()
        alone.append(caches(one))
    assert eng.status() == D.DFLASH_OK
    net = 1e-5 if dtype == "f32" else 2e-2

    def beyond(x, y):  # (codes, exponents) of the same rows: the share of elements beyond the bound
        a, b = values(*x), values(*y)
        size = torch.maximum(a.abs(), b.abs()).amax(-1, keepdim=True)
        scale = torch.exp2(torch.maximum(x[1], y[1]).double() - 127)[..., None]
        tol = (a.abs() + b.abs()) * 2.0 ** -4 / (1 - 2.0 ** -4) + 2 * 2.0 ** -10 * scale + net * size
        return float(((a - b).abs() > tol).double().mean())

    for i, (codes, ex) in enumerate(caches(eng)):
        for s, n in enumerate(LENS):
            mine = codes[s, :, :n], ex[s, :, :n]
            solo = [x[0, :, :n] for x in alone[s][i]]
            assert beyond(mine, solo) == 0.0, (i, s)
            if i % w.target.layers == 0:
                assert torch.equal(mine[0], solo[0]) and torch.equal(mine[1], solo[1]), (i, s)
            other = (s + 1) % 3
            m = min(n, LENS[other])
            assert beyond([x[:, :m] for x in mine], [x[0, :, :m] for x in alone[other][i]]) > 0.25, (i, s)
