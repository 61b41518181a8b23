"""Host-side checks of the operators around the expert layer (no GPU): every refusal is made before any
device is touched, with its status and, for the Python binding, its exception."""
import ctypes

import pytest

OK, INVALID, SHAPE, WS_SMALL, MISALIGNED, NO_DEVICE = 0, 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def m():
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    import nvfp4_w4a4_mixture_gb300 as m

    m.lib()
    return m


def p(addr):
    return None if addr is None else ctypes.c_void_p(addr)


MB = 1 << 20


def norm(m, T=4, H=2048, w_post=40 * MB, w_pre=41 * MB, eps=1e-6, res_type=0, gate=None, gate_type=0, per_channel=1,
         gate_ld=0, y=MB, ld_y=2048, r=2 * MB, ld_r=2048, ro=3 * MB, ld_ro=2048, x=4 * MB, ld_x=2048):
    d = m.NormDesc(H, w_post, w_pre, eps, 0.0, 1.0, res_type, gate, gate_type, per_channel, gate_ld)
    return m.lib().moe_norm_residual(ctypes.byref(d), p(y), ld_y, p(r), ld_r, T, p(ro), ld_ro, p(x), ld_x, None)


def passes(status):
    # every check before the device's passed: refused for want of an sm_103 GPU, or launched where there is one
    return status == NO_DEVICE


@pytest.fixture
def no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses that pass every check: only where nothing can be launched")


def test_norm_refusals(m):
    assert m.lib().moe_norm_residual(None, None, 0, None, 0, 4, None, 0, None, 0, None) == INVALID
    for H in (0, 4, 2049, 8200, -8):
        assert norm(m, H=H) == SHAPE
    assert norm(m, T=-1) == SHAPE
    assert b"T=-1" in m.lib().moe_last_error_detail()
    assert norm(m, res_type=2) == INVALID
    assert norm(m, gate=8 * MB, gate_type=-1) == INVALID
    assert norm(m, eps=-1.0) == INVALID
    assert norm(m, eps=float("nan")) == INVALID
    assert norm(m, y=None, r=None, w_post=None) == INVALID
    assert norm(m, y=None) == INVALID  # w_post without y
    assert norm(m, y=None, w_post=None, gate=8 * MB) == INVALID
    assert norm(m, ro=None, x=None, w_pre=None) == INVALID
    assert norm(m, x=None) == INVALID
    assert norm(m, w_pre=None) == INVALID
    assert norm(m, ld_y=2040) == INVALID
    assert norm(m, y=MB + 2) == MISALIGNED
    assert norm(m, ld_r=2049) == MISALIGNED
    assert norm(m, res_type=1, ld_r=2049, ld_ro=2048) == MISALIGNED
    assert norm(m, w_pre=41 * MB + 8) == MISALIGNED
    assert norm(m, gate=8 * MB + 8) == MISALIGNED
    assert norm(m, gate=8 * MB, gate_ld=-8) == INVALID
    assert norm(m, gate=8 * MB, gate_ld=2044) == MISALIGNED
    assert norm(m, gate=8 * MB + 2, gate_type=1, per_channel=0, gate_ld=1) == MISALIGNED


def test_norm_refuses_overlaps(m):
    row = 2048 * 2
    assert norm(m, x=2 * MB) == INVALID          # x_out on the residual
    assert norm(m, ro=MB) == INVALID             # residual_out on y
    assert norm(m, ro=2 * MB + row) == INVALID   # residual_out a row into the residual
    assert norm(m, ro=2 * MB, ld_ro=4096) == INVALID  # the residual's address with another stride
    assert norm(m, x=3 * MB + 3 * row) == INVALID     # x_out on residual_out's last row
    assert norm(m, w_pre=4 * MB) == INVALID
    assert norm(m, gate=3 * MB) == INVALID


def test_norm_accepts(m, no_gpu):
    row = 2048 * 2
    assert passes(norm(m))
    assert passes(norm(m, ro=2 * MB, x=MB))  # in place
    assert passes(norm(m, x=3 * MB + 4 * row))  # right behind residual_out
    assert passes(norm(m, T=1, ld_y=0, ld_r=0, ld_ro=0, ld_x=0))  # one row: no stride is read
    assert passes(norm(m, y=None, w_post=None, ro=None))
    assert passes(norm(m, r=None))
    assert passes(norm(m, gate=8 * MB + 2, per_channel=0, gate_ld=1))


def test_norm_empty_batch(m):
    assert norm(m, T=0, y=None, r=None, ro=None, x=None) == OK
    assert norm(m, T=0, H=2050) == SHAPE


def select(m, T=4, E=512, k=10, score=1, G=1, keep=1, group_score=1, scale=1.0, bias=None, logits=MB, lt=1, ld=512,
           ids=2 * MB, w=3 * MB):
    d = m.RoutingDesc(E, k, score, G, keep, group_score, 1, scale, bias)
    return m.lib().moe_select_experts(ctypes.byref(d), p(logits), lt, ld, T, p(ids), p(w), None)


def test_select_refusals(m):
    assert m.lib().moe_select_experts(None, None, 1, 0, 0, None, None, None) == INVALID
    for kw in (dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=8, k=9, ld=8), dict(G=0), dict(G=33), dict(G=3),
               dict(G=8, keep=0), dict(G=8, keep=9), dict(E=64, G=16, keep=2, k=9), dict(T=-1)):
        assert select(m, **kw) == SHAPE, kw
    for kw in (dict(score=2), dict(group_score=2), dict(lt=2), dict(logits=None), dict(ids=None), dict(w=None), dict(ld=511),
               dict(ids=MB), dict(w=2 * MB + 4), dict(w=MB + 3 * 512 * 4)):
        assert select(m, **kw) == INVALID, kw
    for kw in (dict(logits=MB + 2), dict(logits=MB + 1, lt=0), dict(ids=2 * MB + 2), dict(w=3 * MB + 1), dict(bias=8 * MB + 2)):
        assert select(m, **kw) == MISALIGNED, kw
    assert select(m, G=8, keep=1, E=64, k=9, ld=64) == SHAPE
    assert b"8 experts in topk_group=1" in m.lib().moe_last_error_detail()


def test_select_accepts(m, no_gpu):
    assert passes(select(m))
    assert passes(select(m, logits=MB + 2, lt=0, ld=513))  # rows need no more than their elements' alignment
    assert passes(select(m, T=1, ld=0))
    assert passes(select(m, E=64, G=16, keep=2, k=8, ld=64))


def test_select_empty_batch(m):
    assert select(m, T=0, logits=None, ids=None, w=None) == OK
    assert select(m, T=0, k=0) == SHAPE


def adapt(m, n=4, r=16, K=2048, N=1024, a=40 * MB, b=41 * MB, scale=42 * MB, x=MB, ld_x=2048, T=4, off=43 * MB, ids=44 * MB,
          S=2, y=2 * MB, ld_y=1024, out=3 * MB, ld_out=1024, ws=50 * MB, ws_bytes=4096):
    d = m.AdaptersDesc(n, r, K, N, a, b, scale)
    return m.lib().moe_adapter_add(ctypes.byref(d), p(x), ld_x, T, p(off), p(ids), S, p(y), ld_y, p(out), ld_out, p(ws),
                                   ws_bytes, None)


def test_adapter_refusals(m):
    assert m.lib().moe_adapter_add(None, None, 0, 4, None, None, 1, None, 0, None, 0, None, 0, None) == INVALID
    for kw in (dict(n=0), dict(r=0), dict(r=12), dict(r=136), dict(K=4), dict(K=2052), dict(K=16392), dict(N=0), dict(N=1028),
               dict(T=-1), dict(S=-1)):
        assert adapt(m, **kw) == SHAPE, kw
    for kw in (dict(S=0), dict(a=None), dict(b=None), dict(scale=None), dict(x=None), dict(off=None), dict(ids=None), dict(y=None),
               dict(out=None), dict(ld_x=2040), dict(ld_y=1016), dict(ld_out=1016), dict(out=MB), dict(out=2 * MB + 2048),
               dict(out=2 * MB, ld_out=2048), dict(ws=None)):
        assert adapt(m, **kw) == INVALID, kw
    for kw in (dict(a=40 * MB + 8), dict(b=41 * MB + 2), dict(scale=42 * MB + 2), dict(off=43 * MB + 2), dict(ids=44 * MB + 1),
               dict(x=MB + 8), dict(ld_x=2052), dict(ld_out=1028), dict(ws=50 * MB + 16)):
        assert adapt(m, **kw) == MISALIGNED, kw
    assert adapt(m, ws_bytes=128) == WS_SMALL


def test_adapter_accepts(m, no_gpu):
    assert passes(adapt(m))
    assert passes(adapt(m, out=2 * MB))  # in place
    assert passes(adapt(m, T=1, ld_x=0, ld_y=0, ld_out=0))


def test_adapter_empty_batch(m):
    assert adapt(m, T=0, S=0, x=None, y=None, out=None, off=None, ids=None, a=None, ws=None) == OK
    assert adapt(m, T=0, r=4) == SHAPE


def test_binding_refuses_other_types_and_shapes(m):
    import torch

    bf = torch.bfloat16
    y = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(TypeError, match="CUDA"):
        m.moe_norm_residual(y, y, w_pre=torch.zeros(64, dtype=bf))
    with pytest.raises(TypeError, match="bf16 or fp32"):
        m.moe_norm_residual(y, y.half())
    with pytest.raises(ValueError, match="both None"):
        m.moe_norm_residual(None, None)
    with pytest.raises(TypeError, match="CUDA"):
        m.moe_select_experts(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="CUDA"):
        m.moe_adapter_add(y, y, torch.zeros(1, 8, 64, dtype=bf), torch.zeros(1, 64, 8, dtype=bf), torch.ones(1),
                          torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1, dtype=torch.int32), ws=m)
