"""GPU: moe_read_device_status() without a workspace reads what calls on every stream have reported, also those still under way."""
import pytest
import torch

from test_attention_ops import Batch, BF, ints, m  # noqa: F401

pytestmark = pytest.mark.gpu


def batch():
    b = Batch(50, [1, 1], [40, 50], 1, 64, 16).fill()
    q, k, v = (b.normal(2, 1, 64).to(BF) for _ in range(3))
    return b, q, k, v


@pytest.mark.parametrize("call", ["attention", "append"])
@pytest.mark.parametrize("others", [0, 2])
def test_a_call_on_another_stream_is_waited_for(m, call, others):  # noqa: F811
    b, q, k, v = batch()
    m._attention_ws.clear()
    good = m.moe_cache_append if call == "append" else m.moe_paged_attention
    args = (None, k, v) if call == "append" else (q,)
    for _ in range(others):  # streams that have called before
        with torch.cuda.stream(torch.cuda.Stream()):
            good(*args, b.k_cache, b.v_cache, *b.tables())
    torch.cuda.synchronize()
    m.moe_read_device_status()
    side, bad = torch.cuda.Stream(), ints([40, -1])
    with torch.cuda.stream(side):
        good(*args, b.k_cache, b.v_cache, *b.tables())  # (its workspace is there)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        good(*args, b.k_cache, b.v_cache, b.offsets, bad, b.pages)
    with pytest.raises(m.MoeError, match="kv_len"):
        m.moe_read_device_status()
    m.moe_read_device_status()
    torch.cuda.synchronize()
    m.moe_read_device_status()


def test_a_reading_clears_before_the_next_call(m):  # noqa: F811
    """A call on a stream of its own directly after a reading: its report is not cleared by that reading."""
    b, q, _, _ = batch()
    bad, side = ints([40, -1]), torch.cuda.Stream()
    ws = m.Workspace(m.moe_attention_workspace_bytes(2, 1, 1, 64, 1))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):
            m.moe_paged_attention(q, b.k_cache, b.v_cache, b.offsets, bad, b.pages, ws=ws)
            with pytest.raises(m.MoeError, match="kv_len"):
                m.moe_read_device_status(ws)
        m.moe_read_device_status(ws)


def test_reports_while_a_reading_is_under_way(m):  # noqa: F811
    """Bad pages and bad lengths in turn on a stream of their own, readings from another: no kind of report is lost."""
    b, q, _, _ = batch()
    ws = m.Workspace(m.moe_attention_workspace_bytes(2, 1, 1, 64, 1))
    report = m.Workspace(4096)
    lens, pages = ints([40, -1]), b.pages.clone()
    pages[1, 0] = 10 ** 9
    torch.cuda.synchronize()
    side, out = torch.cuda.Stream(), torch.empty_like(q)

    def call(kv_len, pages):
        d = m.AttentionDesc(1, 1, 0, 0.125, report.address)
        assert m.lib().moe_paged_attention(m._cache_desc(b.k_cache, b.v_cache, None, None), m._requests_desc(b.offsets, kv_len, pages), d,
                                           q.data_ptr(), 64, 2, out.data_ptr(), 64, None, ws.address, ws.nbytes, m._stream()) == 0

    def kinds():
        found = set()
        for _ in range(3):
            try:
                m.moe_read_device_status(report)
            except m.MoeError as e:
                found |= {k for k in ("kv_len", "page outside") if k in str(e)}
        return found

    for i in range(100):
        with torch.cuda.stream(side):
            call(b.kv_len, pages)  # a page
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2000 * (i % 20))
            call(lens, b.pages)  # a length, some time during the readings
        found = kinds()
        torch.cuda.synchronize()
        found |= kinds()
        assert "kv_len" in found, i  # (it is named first where both are read together)
