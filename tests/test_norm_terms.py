"""GPU: a term of the residual sum that is left out adds nothing, whatever its scale."""
import pytest
import torch

from test_block_ops import BF, gen, moe, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.5, float("inf"), float("nan")])
@pytest.mark.parametrize("T,H", [(4, 2048), (700, 264)])
def test_scale_of_no_residual(moe, T, H, scale):  # noqa: F811
    g = gen(T)
    y, w = randn(g, T, H, dtype=BF), randn(g, H, dtype=BF)
    want = moe.moe_norm_residual(y, torch.zeros_like(y), w_post=w, w_pre=w)
    got = moe.moe_norm_residual(y, None, w_post=w, w_pre=w, residual_scale=scale)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
