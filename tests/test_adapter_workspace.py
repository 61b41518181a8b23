"""GPU: the workspace that moe_adapter_add uses where none is given stays in place, so that its reports are not lost and a
captured call may be replayed, whatever other calls need in between."""
import pytest
import torch

from test_block_ops import BF, adapter_case, check_adapter, moe  # noqa: F401

pytestmark = pytest.mark.gpu


def grow_default_workspace(moe):
    """A router call that needs more scratch than the default workspace has."""
    H, E, k = 256, 64, 6
    dummy = (torch.zeros(1, 1, 8, dtype=torch.uint8, device="cuda"),) * 2 + (torch.ones(1, 2, device="cuda"),)
    layer = moe.MoeLayer(H, E, k, 128, torch.randn(E + 1, H, device="cuda").to(BF), dummy, dummy,
                         torch.ones(E + 1, device="cuda"), prepacked=True)
    T = 64
    while layer.workspace_bytes(T) <= moe._ws(4096).nbytes:
        T *= 2
    before = moe._ws(4096)
    moe.moe_route_topk(torch.randn(T, H, device="cuda").to(BF), layer)
    assert moe._ws(4096) is not before


def test_report_outlives_other_calls(moe):  # noqa: F811
    moe.moe_read_device_status()
    c = adapter_case([3, 200], [0, 7], 2, 16, 256, 256)  # adapter 7 of 2
    moe.moe_adapter_add(**c)
    grow_default_workspace(moe)
    with pytest.raises(moe.MoeError, match="seg_adapter"):
        moe.moe_read_device_status()
    moe.moe_read_device_status()


@pytest.mark.parametrize("lens", [[3, 2], [700, 300]])
def test_captured_call_outlives_other_calls(moe, lens):  # noqa: F811
    c = adapter_case(lens, [0, 1], 2, 64, 2048, 2048)
    want, out = check_adapter(moe, c), torch.zeros_like(c["y"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapter_add(**c, out=out)
    grow_default_workspace(moe)
    filler = [torch.full((4096,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(64)]  # what was given back is used again
    graph.replay()
    moe.moe_read_device_status()
    assert torch.equal(out, want) and all(bool((f == 0x7F).all()) for f in filler)
    c["seg_adapter"][1] = -9
    graph.replay()
    with pytest.raises(moe.MoeError, match="seg_adapter"):
        moe.moe_read_device_status()
    assert all(bool((f == 0x7F).all()) for f in filler)


def test_first_call_of_all_in_a_capture(moe, monkeypatch):  # noqa: F811
    c = adapter_case([700, 300], [0, 1], 2, 64, 2048, 2048)
    want, out = check_adapter(moe, c), torch.zeros_like(c["y"])
    monkeypatch.setattr(moe, "_adapter_ws", {})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapter_add(**c, out=out)
    assert torch.equal(moe.moe_adapter_add(**c), want)  # eager, before any replay
    graph.replay()
    graph.replay()
    moe.moe_read_device_status()
    assert torch.equal(out, want)
