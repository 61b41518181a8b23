"""Whole numbers that moe_paged_attention and its workspace size are given: of any integer type, past 32 bits refused."""
import numpy as np
import pytest
import torch

from test_attention_refusals import m  # noqa: F401


@pytest.mark.parametrize("at", range(5))
def test_workspace_bytes_past_32_bits(m, at):  # noqa: F811
    sizes = [4, 16, 2, 128, 1]
    want = m.moe_attention_workspace_bytes(*sizes)
    assert want and m.moe_attention_workspace_bytes(*(np.int64(v) for v in sizes)) == want
    for far in (1 << 32, -(1 << 32), 1 << 80):
        assert m.moe_attention_workspace_bytes(*sizes[:at], sizes[at] + far, *sizes[at + 1:]) == 0


def test_workspace_bytes_of_other_than_integers(m):  # noqa: F811
    with pytest.raises(TypeError):
        m.moe_attention_workspace_bytes(4, 16, 2, 128, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("marshalled", [True, False])
def test_integers_of_any_type(m, monkeypatch, marshalled):  # noqa: F811
    from test_attention_ops import BF, Batch

    if not marshalled:
        monkeypatch.setattr(m, "_calls", None)
    b = Batch(55, [2, 1], [40, 500], 2, 64, 16).fill()
    q = b.normal(3, 4, 64).to(BF)
    want = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, window=100)
    monkeypatch.setattr(m, "_attention_bytes", {})
    got = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=np.int64(2), window=np.int32(100))
    assert torch.equal(got, want)
    for wrong in (dict(max_new=(1 << 32) + 2), dict(max_new=2, window=1 << 32), dict(max_new=0), dict(max_new=2, window=-1)):
        with pytest.raises((ValueError, m.MoeError)):
            m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), **wrong)
    for wrong in (dict(max_new=2.0), dict(max_new=2, window=1.5)):
        with pytest.raises(TypeError):
            m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), **wrong)
