"""Host-side: the most requests of a batch (no GPU)."""
import pytest

from test_attention_refusals import INVALID, MB, SHAPE, append, attend, m, requests  # noqa: F401


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("S", [(1 << 30) + 1, (1 << 31) - 1])
def test_more_requests_than_are_counted(m, call, S):  # noqa: F811
    R = requests(m, S=S, off=1 << 40, lens=2 << 40, pages=3 << 40)
    assert call(m, R=R) == SHAPE and b"2^30" in m.lib().moe_last_error_detail()
    assert m.moe_attention_workspace_bytes(S, 4, 2, 128, 1) == 0


@pytest.mark.parametrize("call", [append, attend])
def test_the_most_requests(m, call):  # noqa: F811
    R = requests(m, S=1 << 30, off=1 << 40, lens=2 << 40, pages=3 << 40)
    assert call(m, R=R, ws=None) == INVALID and b"workspace" in m.lib().moe_last_error_detail()
    assert m.moe_attention_workspace_bytes(1 << 30, 4, 2, 128, 1) > 8 << 30
