"""Pins of the plain tree-verification reference the GPU tests compare with."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R


def test_e4m3_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.E4M3, t)


def test_quantise_row_properties():
    rng = np.random.default_rng(0)
    for scale in (1e-22, 1e-6, 1.0, 300.0, 1e21):
        x = rng.standard_normal(64) * scale
        c, e = R.quantise_row(x)
        y = R.value_rows(c, np.array(e))
        mx = np.abs(x).max()
        if 448 * 2.0 ** -60 < mx <= 448 * 2.0 ** 60:
            assert 224 * 2.0 ** (e - 127) < mx <= 448 * 2.0 ** (e - 127)
            # half a step: 2^-4 relative, 2^-10 of the scale among the subnormals
            assert (np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e - 127 - 10))).all()
    c, e = R.quantise_row([0.0, -0.0])
    assert e == 127 - 60 and list(c) == [0, 128]
    c, e = R.quantise_row([np.nan, np.inf, -1.75])
    assert list(c[:2]) == [127, 127] and R.value_rows(c, np.array(e))[2] == -1.75


def test_sees():
    assert R.sees([-1, 0, 0, 2, R.PAD, 4, -1]) == [{0}, {0, 1}, {0, 2}, {0, 2, 3}, None, None, {6}]


def test_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v, kb, vb = (rng.standard_normal(s) for s in ((3, 2, 8), (1, 5, 8), (1, 5, 8), (3, 1, 8), (3, 1, 8)))
    out, _, _ = R.attention(q, k, v, kb, vb, [-1, 0, 1], 0.3)
    m = torch.ones(3, 8, dtype=torch.bool)
    m[:, 5:] = torch.tril(torch.ones(3, 3, dtype=torch.bool))
    K, W = torch.tensor(np.concatenate([k[0], kb[:, 0]])), torch.tensor(np.concatenate([v[0], vb[:, 0]]))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q).transpose(0, 1), K.expand(2, 8, 8),
                                                           W.expand(2, 8, 8), attn_mask=m, scale=0.3)
    np.testing.assert_allclose(out, ref.transpose(0, 1).numpy(), atol=1e-13)


@pytest.mark.parametrize("drawn", [False, True])
def test_accept_keeps_the_targets_distribution(drawn):
    """The first emitted token follows softmax(target / T) whatever the
    candidates: 40000 walks over a star of three children, V = 5."""
    rng = np.random.default_rng(3)
    V, T, n = 5, 0.9, 40000
    target, draft = rng.standard_normal((4, V)) * 1.2, rng.standard_normal((1, V)) * 1.2
    p, q = R.softmax(target[0], T), R.softmax(draft[0], T)
    count = np.zeros(V)
    for _ in range(n):
        kids = rng.choice(V, 3, replace=False, p=q) if drawn else np.array([4, 0, 2])
        (k, _, out, _), _ = R.accept([-1, 0, 0, 0], [0, *kids], target, draft if drawn else None, rng.random(4),
                                     rng.exponential(size=V), T, 1)
        count[out[0]] += 1
    # five standard deviations of a binomial share
    np.testing.assert_array_less(np.abs(count / n - p), 5 * np.sqrt(p * (1 - p) / n))
