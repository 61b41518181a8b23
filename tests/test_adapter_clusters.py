"""GPU: adapters whose tiles are shared by a cluster of CTAs. Where K has fewer slices than the cluster has CTAs, some
CTAs have nothing to sum and send their part to the others' shared memory as the first thing they do, which has to wait
until those have started."""
import pytest
import torch

from test_block_ops import adapter_case, check_adapter, moe, randn, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,r,K,N", [([1], 128, 8, 16384), ([4], 128, 32, 16384), ([3, 1, 5], 128, 72, 8192),
                                        ([1, 1], 64, 2048, 2048), ([8] * 9, 128, 40, 4096)])
def test_sums_of_a_cluster_whose_parts_come_at_once(moe, lens, r, K, N):  # noqa: F811
    c = adapter_case(lens, [i % 2 for i in range(len(lens))], 2, r, K, N)
    want = check_adapter(moe, c).clone()
    out, busy = torch.empty_like(want), randn(gen(1), 1024, 1024)
    side = torch.cuda.Stream()
    same = torch.ones((), dtype=torch.bool, device="cuda")
    torch.cuda.synchronize()
    for i in range(200):
        out.fill_(7.0)
        if i % 2:
            with torch.cuda.stream(side):  # work that holds some of the multiprocessors while the clusters start
                busy = busy @ busy * 1e-3
        moe.moe_adapter_add(**c, out=out)
        same &= (out == want).all()
    torch.cuda.synchronize()
    moe.moe_read_device_status()
    assert bool(same)
