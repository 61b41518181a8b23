"""Integers past 32 bits among the selection's arguments are refused by both marshallings, not cut (no GPU)."""
import pytest
import torch

from test_block_refusals import FakeTensor, calls, m  # noqa: F401


def args(**kw):
    a = dict(k=3, score=1, n_group=4, topk_group=2, group_score=1)
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [dict(k=(1 << 32) + 3), dict(score=1 << 32), dict(n_group=(1 << 32) + 4), dict(topk_group=-(1 << 32) + 2),
                                dict(group_score=1 << 31), dict(n_group=1 << 80)])
def test_c_marshalling_leaves_them(calls, kw):  # noqa: F811
    calls, got = calls
    a = args(**kw)
    l, ids, w = FakeTensor(torch.float32, (5, 16), 20), FakeTensor(torch.int32, (5, 3), 21), FakeTensor(torch.float32, (5, 3), 22)
    assert calls.select_experts(l, a["k"], None, a["score"], a["n_group"], a["topk_group"], a["group_score"], True, 1.0, ids, w, 0) == -1
    assert not got


@pytest.mark.parametrize("kw", [dict(k=(1 << 32) + 3), dict(score=1 << 32), dict(n_group=(1 << 32) + 4), dict(topk_group=-(1 << 32) + 2),
                                dict(group_score=1 << 31), dict(n_group=1 << 80)])
def test_binding_refuses_them(m, monkeypatch, kw):  # noqa: F811
    a = args(**kw)
    monkeypatch.setattr(m, "_calls", None)
    monkeypatch.setattr(m, "_stream", lambda: None)
    l, w = FakeTensor(torch.float32, (5, 16), 20), FakeTensor(torch.float32, (5, a["k"]), 22)
    with pytest.raises(ValueError, match="32 bits"):
        m.moe_select_experts(l, out=(FakeTensor(torch.int32, (5, a["k"]), 21), w), **a)
