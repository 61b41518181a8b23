"""GPU: a wait of the adapter kernel that runs out, without a fault. The workspace's test hook makes the MMA warps wait for a
barrier that nobody arrives at, with a 20 ms limit; every other role then waits for what does not come, gives up after
its own limit (1 s), and the kernel drains its copies and products, frees the tensor memory and returns. The status says
so, and the next calls on the same workspace are right."""
import time

import pytest
import torch

from test_block_ops import adapter_case, check_adapter, moe  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,r", [([16384 // 24] * 24, 64),         # one CTA a tile of 128 rows, several tiles a CTA
                                    ([70, 50, 33] * 27, 40),          # one CTA a tile of 64 rows
                                    ([5000], 64), ([1500, 900], 64), ([400, 300], 128)])  # clusters
def test_wait_that_runs_out(moe, lens, r):  # noqa: F811
    c = adapter_case(lens, [i % 2 for i in range(len(lens))], 2, r, 2048, 2048)
    want = check_adapter(moe, c)
    ws = moe.Workspace(4096)
    moe.moe_set_wait_test_hook(ws, 20_000, 1)
    torch.cuda.synchronize()
    start = time.monotonic()
    moe.moe_adapter_add(**c, ws=ws)
    with pytest.raises(moe.MoeError, match="adapter wait timed out"):
        moe.moe_read_device_status(ws=ws)
    assert 0.02 < time.monotonic() - start < 10.0
    moe.moe_set_wait_test_hook(ws, 0, 0)
    for _ in range(3):
        assert torch.equal(moe.moe_adapter_add(**c, ws=ws), want)
    moe.moe_read_device_status(ws=ws)
