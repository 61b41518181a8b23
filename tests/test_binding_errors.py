"""An integer past 32 bits stays an error when a tensor's own methods raise and catch one of their own (no GPU)."""
import torch

from test_block_refusals import FakeTensor, calls, m  # noqa: F401


class Busy(FakeTensor):
    def is_contiguous(self):
        try:
            raise KeyError
        except KeyError:
            return True


def test_the_first_error_stays(calls):  # noqa: F811
    calls, got = calls
    l, ids, w = FakeTensor(torch.float32, (5, 16), 20), Busy(torch.int32, (5, 3), 21), FakeTensor(torch.float32, (5, 3), 22)
    assert calls.select_experts(l, (1 << 32) + 3, None, 1, 4, 2, 1, True, 1.0, ids, w, 0) == -1
    assert not got
