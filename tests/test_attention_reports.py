"""GPU: what moe_paged_attention reports from captured calls, and what a captured call consists of."""
import pytest
import torch

from test_attention_ops import BF, Batch, ints, m  # noqa: F401

pytestmark = pytest.mark.gpu


def test_captured_calls_report_their_tables(m):  # noqa: F811
    b = Batch(51, [1, 2, 1], [40, 500, 60], 2, 64, 16).fill()
    q = b.normal(4, 4, 64).to(BF)
    call = lambda out: m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=out)  # noqa: E731
    want = call(torch.empty_like(q))
    m.moe_read_device_status()
    outs, graphs = [torch.empty_like(q) for _ in range(2)], []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append(g)

    def replay():
        for out, g, s in zip(outs, graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
            out.fill_(7.0)
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                g.replay()

    replay()
    m.moe_read_device_status()
    assert all(torch.equal(out, want) for out in outs)
    lens, pages = b.kv_len.clone(), b.pages.clone()
    b.kv_len.copy_(ints([40, -3, 60]))
    replay()
    with pytest.raises(m.MoeError, match="kv_len"):
        m.moe_read_device_status()
    assert all(torch.equal(out[0], want[0]) and bool((out[1:3] == 7.0).all()) and torch.equal(out[3], want[3]) for out in outs)
    b.kv_len.copy_(lens)
    b.pages[1, 2] = 10 ** 9
    replay()
    with pytest.raises(m.MoeError, match="page outside"):
        m.moe_read_device_status()
    b.pages.copy_(pages)
    replay()
    m.moe_read_device_status()
    assert all(torch.equal(out, want) for out in outs)


def test_scratch_holds_anything_before_a_call(m, monkeypatch):  # noqa: F811
    """Scratch whose memory held other values: nothing of it is read before it is written, its header neither."""
    b = Batch(52, [1, 2, 1], [9000, 500, 60], 2, 128, 16).fill()
    q = b.normal(4, 8, 128).to(BF)
    want = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2)
    made = m.Workspace

    class Filled(made):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            if kw.get("cleared") is False:
                self.tensor.fill_(0x7F)

    monkeypatch.setattr(m, "Workspace", Filled)
    monkeypatch.setattr(m, "_attention_ws", {})
    assert torch.equal(m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2), want)
    out, graph = torch.empty_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    m.moe_read_device_status()


def test_first_call_of_all_in_a_capture(m, monkeypatch):  # noqa: F811
    b = Batch(53, [1, 2], [3000, 500], 2, 128, 16).fill()
    q = b.normal(3, 8, 128).to(BF)
    want, out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2), torch.empty_like(q)
    monkeypatch.setattr(m, "_adapter_ws", {})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=out)
    assert not m._adapter_ws
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_a_report_of_ones_own(m):  # noqa: F811
    """The C call with a report beside the workspace: its status word is the one that is set and read."""
    b = Batch(54, [1, 1], [40, 50], 1, 64, 16).fill()
    q, out = b.normal(2, 1, 64).to(BF), torch.empty(2, 1, 64, dtype=BF, device="cuda")
    ws, report = m.Workspace(m.moe_attention_workspace_bytes(2, 1, 1, 64, 1)), m.Workspace(4096)
    bad = ints([40, -1])
    d = m.AttentionDesc(1, 1, 0, 0.125, report.address)
    status = m.lib().moe_paged_attention(m._cache_desc(b.k_cache, b.v_cache, None, None), m._requests_desc(b.offsets, bad, b.pages), d,
                                         q.data_ptr(), 64, 2, out.data_ptr(), 64, None, ws.address, ws.nbytes, m._stream())
    assert status == 0
    m.moe_read_device_status(ws)
    with pytest.raises(m.MoeError, match="kv_len"):
        m.moe_read_device_status(report)
    m.moe_read_device_status(report)
