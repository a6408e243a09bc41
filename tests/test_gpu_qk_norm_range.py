"""dflash_qk_norm_rope at the ends of the range of sizes that it takes."""
import pytest
import torch

from tests import test_gpu_qk_norm as Q

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,src", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("size", [2.0 ** 59, 2.0 ** -50])
def test_sizes_of_heads(monkeypatch, dtype, src, d, eps, size):
    """Every head's largest element has that size, or nearly."""
    monkeypatch.setattr(Q, "EPS", eps)
    p = Q.Heads([10, 20], 5, d=d, dtype=dtype, src=src, seed=3)
    x = p.qkv[:, :p.width].double().view(p.M, -1, d)
    x = x / x.abs().amax(-1, keepdim=True) * size
    if size < 1:  # (none is much smaller)
        x = torch.where(x.abs() < size / 2, x.sign() * size / 2, x)
    p.qkv[:, :p.width] = x.view(p.M, -1).to(p.qkv.dtype)
    p.run()
    p.check()
