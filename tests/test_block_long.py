"""Block operators where numbers pass 32 bits: tokens, and offsets of elements and bytes."""
import pytest
import torch

from test_block_ops import BF, adapter_case, check_adapter, gen, moe, randn  # noqa: F401
from test_block_refusals import FakeTensor, m  # noqa: F401


def test_more_rows_than_the_calls_count_are_refused(m):  # noqa: F811
    for T in (1 << 31, (1 << 32) + 4):
        with pytest.raises(ValueError, match="2147483647"):
            m._rows(FakeTensor(BF, (T, 8), 1), "y", BF, (T, 8))
        with pytest.raises(ValueError, match="2147483647"):
            m._whole(FakeTensor(torch.int32, (T,), 1), "seg_adapter", torch.int32, (T,))
    T = (1 << 31) - 1
    assert m._rows(FakeTensor(BF, (T, 8), 1), "y", BF, (T, 8)) == (1, 8)


@pytest.mark.gpu
def test_selection_of_as_many_tokens_as_the_call_counts(moe):  # noqa: F811
    T = (1 << 31) - 1
    l = torch.zeros(T, 1, dtype=BF, device="cuda")
    l[-1], l[-2] = float("-inf"), 3.0
    ids, w = moe.moe_select_experts(l, 1, renormalize=False, scale=0.5)
    assert int(ids.max()) == 0 and int(ids.min()) == 0
    assert w[-4:].flatten().tolist() == [0.5, 0.5, 0.5, 0.0] and float(w[:-1].min()) == 0.5 and float(w.max()) == 0.5


@pytest.fixture
def far():
    """Rows of the given values 2^29 elements and more apart: the last of nine starts past 2^32 elements."""
    def place(t):
        ld = (1 << 29) + 8
        buf = torch.empty(ld * (t.shape[0] - 1) + t.shape[1], dtype=t.dtype, device="cuda")
        view = buf.as_strided(t.shape, (ld, 1))
        view.copy_(t)
        return view

    yield place
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_rows_far_apart(moe, far):  # noqa: F811
    g = gen(4)
    T, H = 9, 520
    y, r, w = randn(g, T, H, dtype=BF), randn(g, T, H), randn(g, H, dtype=BF)
    want = moe.moe_norm_residual(y, r, w_post=w, w_pre=w)
    got = far(torch.zeros_like(r)), far(torch.zeros_like(y))
    moe.moe_norm_residual(far(y), far(r), w_post=w, w_pre=w, out=got)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del got
    for dtype in (torch.float32, BF):
        l = randn(g, T, 256, dtype=dtype)
        want, got = moe.moe_select_experts(l, 8), moe.moe_select_experts(far(l), 8)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c = adapter_case([5, 1, 3], [0, -1, 1], 2, 24, H, 264)
    want, got = moe.moe_adapter_add(**c), far(torch.zeros_like(c["y"]))
    moe.moe_adapter_add(**dict(c, x=far(c["x"]), y=far(c["y"])), out=got)
    assert torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("r", [16, 64])
def test_long_batches(moe, r):  # noqa: F811
    # outputs of 2^31 elements and more, through the kernel of long requests
    T, K, N = 150000, 64, 16384
    c = adapter_case([T - 5, 5], [0, 1], 2, r, K, N)
    got = moe.moe_adapter_add(**c)
    moe.moe_read_device_status()
    for rows in (slice(0, 300), slice(131072 - 100, 131072 + 100), slice(T - 300, T)):  # 131,072 rows are 2^31 elements
        lens = [rows.stop - rows.start - 5, 5] if rows.stop == T else [rows.stop - rows.start, 0]
        part = dict(c, x=c["x"][rows], y=c["y"][rows],
                    seg_offsets=torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda"))
        # the split of the sums over K goes by the batch: equal up to a step of bf16, each result being its own rounding
        want = moe.moe_adapter_add(**part)
        assert float((got[rows].double() - want.double()).norm()) <= 2.0 ** -8 * float(want.double().norm())
        assert torch.all((got[rows].double() - want.double()).abs() <= 2.0 ** -7 * (want.double().abs() + 1e-2))


@pytest.mark.gpu
def test_norms_of_a_long_batch(moe):  # noqa: F811
    g = gen(8)
    T, H = 270000, 8192
    y, r, w = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda"), randn(g, H, dtype=BF)
    y.normal_(generator=g), r.normal_(generator=g)
    got = moe.moe_norm_residual(y, r, w_post=w, w_pre=w)
    for rows in (slice(0, 400), slice(262144 - 200, 262144 + 200), slice(T - 400, T)):  # 262,144 rows are 2^31 elements
        want = moe.moe_norm_residual(y[rows], r[rows], w_post=w, w_pre=w)
        assert torch.equal(got[0][rows], want[0]) and torch.equal(got[1][rows], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,r,K,N", [([5, 1], 128, 16384, 16384), ([700, 300], 128, 16384, 1024), ([5000], 64, 1024, 16384),
                                        ([70, 50, 33] * 27, 40, 16384, 520)])
def test_adapters_of_the_largest_widths(moe, lens, r, K, N):  # noqa: F811
    check_adapter(moe, adapter_case(lens, [i % 2 for i in range(len(lens))], 2, r, K, N))
