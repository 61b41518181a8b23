"""GPU: a bounded wait of the FP8 product and of the attention that runs out (by the workspace's test hook, without a fault) is
reported, the launch ends by itself, and the next call on the same workspace is as if nothing had been."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    import nvfp4_w4a4_mixture_gb300 as m

    return m


def run_out(m, ws, call):
    want = call()
    m.moe_read_device_status(ws)
    m.moe_set_wait_test_hook(ws, 1000, 1)
    call()
    with pytest.raises(m.MoeError) as e:
        m.moe_read_device_status(ws)
    assert e.value.status == "MOE_ERR_DEVICE_TIMEOUT" or "timed out" in str(e.value)
    m.moe_set_wait_test_hook(ws, 0, 0)
    assert torch.equal(call(), want)
    m.moe_read_device_status(ws)


@pytest.mark.parametrize("T,N,K", [(4, 512, 1024), (40, 256, 2048), (300, 2048, 512)])
def test_gemm_fp8(m, T, N, K):
    g = torch.Generator(device="cuda").manual_seed(T)
    a, b = (torch.randn(n, K, generator=g, device="cuda").to(torch.float8_e4m3fn) for n in (T, N))
    sa, sb = torch.ones(T, K // 128, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
    ws = m.Workspace(4096)
    run_out(m, ws, lambda: m.moe_gemm_fp8(a, sa, b, sb, ws=ws))


@pytest.mark.parametrize("new,n_q", [(1, 4), (2, 32)])
def test_attention(m, new, n_q):
    g = torch.Generator(device="cuda").manual_seed(new)
    k, v = (torch.randn(40, 16, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2 * new, n_q, 64, generator=g, device="cuda").to(torch.bfloat16)
    off, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new, 2 * new], [300, 77]))
    pages = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    ws = m.Workspace(m.moe_attention_workspace_bytes(2, n_q, 2, 64, new))
    run_out(m, ws, lambda: m.moe_paged_attention(q, k, v, off, lens, pages, max_new=new, ws=ws))
