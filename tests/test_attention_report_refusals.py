"""Host-side checks of moe_attention_t.report (no GPU)."""
import ctypes

from test_attention_refusals import INVALID, MB, MISALIGNED, NO_DEVICE, cache, m, no_gpu, p, requests  # noqa: F401


def attend(m, report):  # noqa: F811
    d = m.AttentionDesc(4, 1, 0, 0.1, report)
    return m.lib().moe_paged_attention(ctypes.byref(cache(m)), ctypes.byref(requests(m)), ctypes.byref(d), p(MB), 512, 4, p(4 * MB), 512,
                                       None, p(300 * MB), 1 << 30, None)


def test_report(m):  # noqa: F811
    assert attend(m, 500 * MB + 128) == MISALIGNED
    assert m.AttentionDesc(4, 1, 0, 0.1).report is None
    for at in (300 * MB + 256, 300 * MB + (1 << 30) - 256):  # in the call's scratch
        assert attend(m, at) == INVALID and b"report" in m.lib().moe_last_error_detail()


def test_taken(m, no_gpu):  # noqa: F811
    for at in (None, 300 * MB, 300 * MB - 256, 300 * MB + (1 << 30)):
        assert attend(m, at) == NO_DEVICE
