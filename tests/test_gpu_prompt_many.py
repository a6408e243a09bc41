"""Packed prompts of tens of thousands of sequences."""
import pytest
import torch

from block_diffusion_speculative_step_gb300 import dflash as D
from tests.prompt_ref import FILL, Prompt

pytestmark = pytest.mark.gpu

DTYPES = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
def test_as_many_as_a_call_takes(dtype):
    """65536 sequences of one row over nothing: a row sees itself alone."""
    p = Prompt([1] * 65536, 4, 2, 64, dtype, lead=3, tail=9, seed=50)
    p.run()
    torch.cuda.synchronize()
    assert p.ws.status() == D.DFLASH_OK
    got, want = p.out[3:-9].double(), p.vb[3:-9].repeat_interleave(2, 1).double()
    tol = (2.0 ** -16 + 2.0 ** -20) * want.abs() + (torch.finfo(p.dt).eps / 2) * want.abs() * 1.01  # (two terms, the sum's quotient, a half step)
    assert bool(((got - want).abs() <= tol).all())
    assert bool((p.out[:3] == FILL).all()) and bool((p.out[-9:] == FILL).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["empty ones between", "one long"])
def test_thousands_over_contexts(dtype, kind):
    S = 20000
    if kind == "one long":
        lens, ctx = [1] * S, [(3 * i) % 9 for i in range(S)]
        lens[12345], ctx[12345] = 300, 700
    else:
        lens, ctx = [3 if i % 7 == 3 else 0 for i in range(S)], [(5 * i) % 140 for i in range(S)]
    p = Prompt(lens, 4, 2, 64, dtype, ctx=ctx, seed=51)
    p.run()
    p.check(seqs=[i for i in list(range(0, S, 397)) + list(range(12340, 12350)) + [S - 1] if lens[i]])
    assert bool((p.out != FILL).flatten(1).any(1).all())  # every row was written


def test_more_sequences_than_a_call_takes():
    p = Prompt([1] * 10, 4, 2, 64, "bf16")
    p.a.n_seqs = 65537
    with pytest.raises(D.DFlashError) as e:
        p.run()
    assert e.value.code == D.DFLASH_ERR_UNSUPPORTED
