"""GPU: one summing warp of the FP8 product's kernel for few tokens gives up in the middle of its blocks (by the workspace's test
hook, without a fault) while the others go on: the launch ends by itself, no CTA of its cluster stores a sum without that warp's
part, and the next call is as if nothing had been."""
import time

import pytest
import torch

from test_attention_ops import gemm_case, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K,cluster", [(4, 128, 65536, True), (20, 128, 16384, True), (40, 256, 16384, True), (5, 40000, 2048, False)])
def test_one_warp_gives_up(m, T, N, K, cluster):  # noqa: F811
    a, sa, b, sb = gemm_case(T, N, K, T)
    ws = m.Workspace(4096)
    want = m.moe_gemm_fp8(a, sa, b, sb, ws=ws)
    m.moe_read_device_status(ws)
    out = torch.full_like(want, 7.0)
    m.moe_set_wait_test_hook(ws, 1000, 2)
    torch.cuda.synchronize()
    start = time.monotonic()
    m.moe_gemm_fp8(a, sa, b, sb, out=out, ws=ws)
    with pytest.raises(m.MoeError, match="timed out"):
        m.moe_read_device_status(ws)
    assert time.monotonic() - start < 10.0
    if cluster:
        assert bool((out == 7.0).all())
    m.moe_set_wait_test_hook(ws, 0, 0)
    for _ in range(3):
        assert torch.equal(m.moe_gemm_fp8(a, sa, b, sb, ws=ws), want)
    m.moe_read_device_status(ws)
