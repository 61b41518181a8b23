"""Which views of one buffer the block operators take: rows in different columns of it are apart, however their spans lie.
Without a GPU through the C calls with made-up addresses, on one with real views."""
import pytest
import torch

from test_block_ops import adapter_case, check_adapter, gen, moe, randn  # noqa: F401
from test_block_refusals import INVALID, MB, adapt, m, no_gpu, norm, passes, select  # noqa: F401


def test_norm_takes_columns_of_one_buffer(m, no_gpu):  # noqa: F811
    H, b = 2048, 2048 * 2  # elements and bytes of a row
    # residual_out and x_out side by side, and beside the inputs; one starting rows after the other
    assert passes(norm(m, ro=3 * MB, ld_ro=2 * H, x=3 * MB + b, ld_x=2 * H))
    assert passes(norm(m, ro=3 * MB + b, ld_ro=2 * H, x=3 * MB, ld_x=2 * H))
    assert passes(norm(m, y=MB, ld_y=4 * H, r=MB + b, ld_r=4 * H, ro=MB + 2 * b, ld_ro=4 * H, x=MB + 3 * b, ld_x=4 * H))
    assert passes(norm(m, r=2 * MB, ld_r=3 * H, ro=2 * MB, ld_ro=3 * H, x=2 * MB + b + 2 * 3 * b, ld_x=3 * H))
    assert passes(norm(m, res_type=1, r=2 * MB, ld_r=2 * H, ro=2 * MB, ld_ro=2 * H, x=2 * MB + 2 * b, ld_x=4 * H))
    # x_out starts in the gap of residual_out's last row and goes on behind it
    assert passes(norm(m, ro=3 * MB, ld_ro=H + 64, x=3 * MB + 3 * (b + 128) + b, ld_x=H + 64))


def test_norm_refuses_columns_that_meet(m):  # noqa: F811
    H, b = 2048, 2048 * 2
    assert norm(m, ro=3 * MB, ld_ro=2 * H, x=3 * MB + b - 16, ld_x=2 * H) == INVALID
    assert norm(m, ro=3 * MB, ld_ro=2 * H, x=3 * MB + b + 16, ld_x=2 * H) == INVALID  # its end is the next row's start
    assert norm(m, ro=3 * MB, ld_ro=2 * H - 8, x=3 * MB + b, ld_x=2 * H - 8) == INVALID
    assert norm(m, ro=3 * MB + 2 * b, ld_ro=2 * H, x=3 * MB, ld_x=2 * H) == INVALID  # the same columns, one row on
    assert norm(m, ro=3 * MB, ld_ro=2 * H, x=3 * MB + b, ld_x=2 * H + 8) == INVALID  # other strides: by their spans
    assert norm(m, ro=3 * MB, ld_ro=H + 64, x=3 * MB + 2 * (b + 128) + b, ld_x=H + 64) == INVALID


def test_adapter_columns_of_one_buffer(m, no_gpu):  # noqa: F811
    K, N = 2048, 1024
    for x, y, out in ((0, K, K), (N, 0, 0), (0, K, K + N), (2 * N, 0, N), (N, K + N, 0)):
        ld = K + 2 * N
        assert passes(adapt(m, x=MB + 2 * x, ld_x=ld, y=MB + 2 * y, ld_y=ld, out=MB + 2 * out, ld_out=ld))
    assert adapt(m, x=MB, ld_x=K + N, y=2 * MB, out=MB + 2 * (K - 8), ld_out=K + N) == INVALID
    assert adapt(m, x=MB, ld_x=K + N, y=2 * MB, out=MB + 2 * (K + 8), ld_out=K + N) == INVALID
    assert adapt(m, y=2 * MB, ld_y=2 * N, out=2 * MB + 2 * (N - 8), ld_out=2 * N) == INVALID


def test_outputs_on_the_small_inputs_are_refused(m):  # noqa: F811
    # one of T * k ids or weights on one of E biases
    for kw in (dict(bias=2 * MB), dict(bias=3 * MB + 4 * 10 * 4 - 4), dict(bias=2 * MB - 512 * 4 + 4)):
        assert select(m, **kw) == INVALID, kw
    last = 3 * MB + 3 * 1024 * 2 + 1024 * 2  # behind out's last row
    for kw in (dict(a=3 * MB), dict(b=last - 16), dict(scale=last - 4), dict(off=3 * MB + 4), dict(ids=last - 4),
               dict(off=3 * MB - 8), dict(ids=3 * MB - 4), dict(a=3 * MB - 4 * 16 * 2048 * 2 + 16)):
        assert adapt(m, **kw) == INVALID, kw
        assert b"overlap" in m.lib().moe_last_error_detail()


def test_outputs_beside_the_small_inputs(m, no_gpu):  # noqa: F811
    last = 3 * MB + 3 * 1024 * 2 + 1024 * 2
    for kw in (dict(bias=3 * MB + 4 * 10 * 4), dict(bias=2 * MB - 512 * 4)):
        assert passes(select(m, **kw)), kw
    for kw in (dict(b=last), dict(scale=last), dict(off=last), dict(ids=last), dict(off=3 * MB - 12), dict(ids=3 * MB - 8),
               dict(a=3 * MB - 4 * 16 * 2048 * 2)):
        assert passes(adapt(m, **kw)), kw


@pytest.mark.gpu
def test_columns_of_one_buffer_give_the_same(moe):  # noqa: F811
    g = gen(2)
    for T in (5, 700):
        H = 520
        buf = randn(g, T, 4 * H, dtype=torch.bfloat16)
        y, r, r_out, x_out = (buf[:, i * H: (i + 1) * H] for i in range(4))
        w = randn(g, H, mean=1.0, std=0.1, dtype=torch.bfloat16)
        want = moe.moe_norm_residual(y.clone(), r.clone(), w_post=w, w_pre=w)
        moe.moe_norm_residual(y, r, w_post=w, w_pre=w, out=(r_out, x_out))
        assert torch.equal(r_out, want[0]) and torch.equal(x_out, want[1])
        c = adapter_case([T - 3, 3], [1, 0], 2, 24, H, H)
        want = check_adapter(moe, c)
        buf[:, :H], buf[:, H: 2 * H] = c["x"], c["y"]
        c["x"], c["y"] = y, r
        assert torch.equal(moe.moe_adapter_add(**c, out=r_out), want)
        assert torch.equal(moe.moe_adapter_add(**c, out=r), want)
