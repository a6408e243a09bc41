"""dflash_token_logprobs where logits lie further apart than fp32's largest number."""
import pytest
import torch

from tests.test_gpu_logprobs import Scores, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [100, 40000])
@pytest.mark.parametrize("T", [2.5, 100.0, 1e29])
def test_logits_of_either_end(V, T):
    """Their log probability over the temperature is in range."""
    x = rand(4, V, 8)
    x[0, :] = -3.4e38
    x[0, 5] = 3.4e38
    x[1] *= 1e37
    x[2, 7:] = -3.4028234663852886e38
    x[2, :7] = 1e38
    x[3, 3], x[3, 4] = 3e38, -3e38
    p = Scores(x, 8, T=T, tokens=[4, 1, 9, 4])
    p.run()
    p.check()
