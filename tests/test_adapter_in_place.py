"""GPU: adapters added in place again and again, each call reading what the one before it has just written."""
import pytest
import torch

from test_block_ops import adapter_case, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,r,K,N", [([1] * 256, 32, 2048, 2048), ([3, 1], 64, 2048, 2048), ([1, 2, 8, 9] * 10, 16, 264, 520),
                                        ([600, 130, 1], 40, 520, 1032)])
def test_in_place_calls_in_a_row(moe, lens, r, K, N):  # noqa: F811
    c = adapter_case(lens, [(i % 4) - 1 if i else 1 for i in range(len(lens))], 3, r, K, N)
    y = c.pop("y")
    a, b = y.clone(), torch.empty_like(y)
    for _ in range(20):
        moe.moe_adapter_add(y=a, out=b, **c)
        a, b = b, a
    for _ in range(20):
        moe.moe_adapter_add(y=y, out=y, **c)
    moe.moe_read_device_status()
    assert torch.equal(a, y)
