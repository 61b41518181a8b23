"""GPU: adapters added in place again and again, each call reading what the one before it has just written, and rows
without an adapter, which are y's values in every kernel, the sign of a zero included."""
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


@pytest.mark.parametrize("lens,r,K,N", [([1] * 40, 16, 256, 256), ([5000, 9], 64, 2048, 2048), ([3000, 3000], 64, 2048, 2048),
                                        ([40, 130, 7, 64] * 25, 40, 1032, 2056)])
def test_rows_without_adapter_keep_their_values(moe, lens, r, K, N):  # noqa: F811
    c = adapter_case(lens, [-1 if i % 2 == 0 else 0 for i in range(len(lens))], 1, r, K, N)
    c["y"][::3], c["y"][1::7, ::5] = -0.0, float("nan")
    off = c["seg_offsets"].tolist()
    for out in (None, c["y"].clone()):
        y = c["y"] if out is None else out
        want = y.clone()
        got = moe.moe_adapter_add(**dict(c, y=y), out=out)
        for i in range(0, len(lens), 2):
            rows = slice(off[i], off[i + 1])
            real = ~want[rows].isnan()
            assert torch.equal(got[rows].isnan(), ~real)
            assert torch.equal(got[rows].view(torch.int16)[real], want[rows].view(torch.int16)[real])
