"""dflash_prompt_attention with the largest and smallest values that it takes,
under scores of any size: sums of weights times values stay in range, in whole
items, in items of one tile and in joined ones."""
import pytest
import torch

from tests.prompt_ref import Prompt

pytestmark = pytest.mark.gpu

SHAPES = [([300, 64], None), ([2000], None), ([1], [20000]), ([1, 3] * 10, [100 * i for i in range(20)]), ([200], [9000])]


def problem(dtype, lens, ctx, scores, size, spread=1.0):
    """scores: the mean score of (slot or row) number j of a sequence, spread the
    others' part in it; values in [size / 2, size)."""
    p = Prompt(lens, 4, 2, 64, dtype, ctx=ctx, seed=40, q_amp=spread)
    g = torch.Generator(device="cuda").manual_seed(41)
    value = lambda x: ((0.5 + 0.498 * torch.rand(x.shape, generator=g, device="cuda")) * size).to(p.dt)
    p.q[:, :, 0] = 8.0  # (with scale 1 / 8 a key's first element is its score's mean)
    p.vb.copy_(value(p.vb))
    for s, n in enumerate(lens):
        c = ctx[s] if ctx else 0
        mean = scores(torch.arange(c + n, device="cuda").float()).to(p.dt)
        p.kb[p.start[s]:p.start[s + 1], :, 0] = mean[c:, None]
        if c:
            p.kc[s, :, :c, 0] = mean[:c]
            p.vc[s, :, :c] = value(p.vc[s, :, :c])
    return p


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,ctx", SHAPES)
@pytest.mark.parametrize("score", [-40.0, 0.0, 5.0, 10.0, 14.0, 16.0, 20.0, 60.0])
@pytest.mark.parametrize("size", [2.0 ** 88, 2.0 ** -60])
def test_values_at_the_ends_of_their_range(dtype, lens, ctx, score, size):
    p = problem(dtype, lens, ctx, lambda j: torch.full_like(j, score), size)
    p.run()
    p.check()


@pytest.mark.parametrize("lens,ctx", SHAPES)
@pytest.mark.parametrize("kind", ["up", "down", "first", "saw"])
def test_scores_that_change_along_the_keys(lens, ctx, kind):
    """Sums that outgrow the reference by little at a time, or that a few early
    keys fill, which later ones do not reach."""
    scores = {"up": lambda j: j / 64, "down": lambda j: 20 - j / 64, "first": lambda j: torch.where(j < 40, 11.5, -3.0),
              "saw": lambda j: (j % 256) / 16}[kind]
    p = problem("bf16", lens, ctx, scores, 2.0 ** 88)
    p.run()
    p.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,ctx", [([1], [150000]), ([200], [150000]), ([1, 1, 1], [90000, 5, 150000])])
@pytest.mark.parametrize("score", [0.0, 10.0, 16.5])
def test_many_keys_of_one_score(dtype, lens, ctx, score):
    """No key stands out: every chunk adds as much as the one before."""
    p = problem(dtype, lens, ctx, lambda j: torch.full_like(j, score), 2.0 ** 88, spread=0.0)
    p.run()
    p.check()
