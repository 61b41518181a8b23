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


class FakeTensor:
    def __init__(self, dtype, shape, ptr, cuda=True, contiguous=True):
        self.dtype, self.shape, self.ptr, self.is_cuda, self.contiguous = dtype, tuple(shape), ptr, cuda, contiguous

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return self.ptr


@pytest.fixture
def calls(m):
    """The C marshalling bound to functions that record what they are given, and the record."""
    import torch

    if m._calls is None:
        pytest.skip("built without Python's headers")
    c, got = ctypes, []
    vp, i32, i64, sz = c.c_void_p, c.c_int, c.c_int64, c.c_size_t
    fields = lambda d: tuple(getattr(d, n) for n, _ in d._fields_)  # noqa: E731
    proto = (c.CFUNCTYPE(i32, c.POINTER(m.NormDesc), vp, i64, vp, i64, i32, vp, i64, vp, i64, vp),
             c.CFUNCTYPE(i32, c.POINTER(m.RoutingDesc), vp, i32, i64, i32, vp, vp, vp),
             c.CFUNCTYPE(i32, c.POINTER(m.AdaptersDesc), vp, i64, i32, vp, vp, i32, vp, i64, vp, i64, vp, sz, vp))

    def record(d, *rest):
        got.append((fields(d.contents), rest))
        return 2

    fs = [p(record) for p in proto]
    m._calls.bind(*(c.cast(f, vp).value for f in fs), torch.bfloat16, torch.float32, torch.int32)
    yield m._calls, got
    m._load_calls(m.lib())


def test_c_marshalling_passes_what_it_is_given(calls):
    import torch

    calls, got = calls
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    y, r, x = FakeTensor(bf, (4, 64), 10), FakeTensor(f32, (4, 64), 11), FakeTensor(bf, (4, 64), 12)
    w = FakeTensor(bf, (64,), 13)
    gates = {None: (None, 0, 0, 0), FakeTensor(bf, (64,), 14): (14, 0, 1, 0), FakeTensor(f32, (4, 1), 15): (15, 1, 0, 1),
             FakeTensor(bf, (4, 64), 16): (16, 0, 1, 64)}
    for g, (p_, t_, c_, ld_) in gates.items():
        assert calls.norm_residual(y, r, w, w, g, 0.5, 0.25, 1.0, r, x, 99) == 2
        d, rest = got.pop()
        assert d == (64, 13, 13, 0.25, 1.0, 0.5, 1, p_, t_, c_, ld_)
        assert rest == (10, 64, 11, 64, 4, 11, 64, 12, 64, 99)
    assert calls.norm_residual(None, y, None, w, None, 1.0, 0.5, 0.0, y, x, 0) == 2
    assert got.pop() == ((64, None, 13, 0.5, 0.0, 1.0, 0, None, 0, 0, 0), (None, 64, 10, 64, 4, 10, 64, 12, 64, None))
    l, ids, wt, b = FakeTensor(bf, (5, 16), 20), FakeTensor(i32, (5, 3), 21), FakeTensor(f32, (5, 3), 22), FakeTensor(f32, (16,), 23)
    assert calls.select_experts(l, 3, b, 1, 4, 2, 1, True, 2.5, ids, wt, 7) == 2
    assert got.pop() == ((16, 3, 1, 4, 2, 1, 1, 2.5, 23), (20, 0, 16, 5, 21, 22, 7))
    a_, b_, s = FakeTensor(bf, (2, 8, 64), 30), FakeTensor(bf, (2, 32, 8), 31), FakeTensor(f32, (2,), 32)
    off, ad, o = FakeTensor(i32, (4,), 33), FakeTensor(i32, (3,), 34), FakeTensor(bf, (4, 32), 35)
    assert calls.adapter_add(y, o, a_, b_, s, off, ad, o, 36, 4096, 8) == 2
    assert got.pop() == ((2, 8, 64, 32, 30, 31, 32), (10, 64, 4, 33, 34, 3, 35, 32, 35, 32, 36, 4096, 8))
    assert not got


def test_c_marshalling_leaves_the_rest_alone(calls):
    import torch

    calls, got = calls
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    T = FakeTensor

    def norm(y=T(bf, (4, 64), 1), r=T(bf, (4, 64), 2), w=T(bf, (64,), 3), g=None, ro=T(bf, (4, 64), 4), x=T(bf, (4, 64), 5)):
        return calls.norm_residual(y, r, w, w, g, 1.0, 1e-6, 0.0, ro, x, 0)

    assert norm() == 2
    got.clear()
    for kw in (dict(y=T(f32, (4, 64), 1)), dict(y=T(bf, (4, 64), 1, cuda=False)), dict(y=T(bf, (4, 64), 1, contiguous=False)),
               dict(y=T(bf, (4, 72), 1)), dict(y=T(bf, (256,), 1)), dict(r=T(torch.float16, (4, 64), 2)), dict(r=T(f32, (4, 64), 2)),
               dict(w=T(bf, (72,), 3)), dict(w=T(f32, (64,), 3)), dict(g=T(bf, (3, 64), 6)), dict(g=T(torch.float16, (64,), 6)),
               dict(g=T(bf, (1, 64), 6)), dict(ro=None), dict(ro=T(bf, (4, 64), 4, cuda=False)), dict(x=T(bf, (5, 64), 5)), dict(y=3),
               dict(y=T(bf, (1 << 40, 64), 1))):
        assert norm(**kw) == -1, kw
    l, ids, wt = T(f32, (5, 16), 20), T(i32, (5, 3), 21), T(f32, (5, 3), 22)
    for args in ((l, 4, None), (l, 0, None), (l, "3", None), (l, 3, T(bf, (16,), 1)), (T(i32, (5, 16), 20), 3, None)):
        assert calls.select_experts(*args, 1, 1, 1, 0, True, 1.0, ids, wt, 0) == -1, args
    y, a_, b_, s = T(bf, (4, 64), 10), T(bf, (2, 8, 64), 30), T(bf, (2, 64, 8), 31), T(f32, (2,), 32)
    off, ad = T(i32, (4,), 33), T(i32, (3,), 34)
    for args in ((y, y, a_, T(bf, (2, 64, 16), 31), s, off, ad, y), (y, y, a_, b_, s, T(i32, (3,), 33), ad, y),
                 (y, y, T(bf, (2, 8, 72), 30), b_, s, off, ad, y), (y, y, a_, b_, s, off, T(torch.int64, (3,), 34), y),
                 (y, y, a_, b_, s, off, ad, T(bf, (4, 72), 1)), (y, y, a_, b_, T(f32, (3,), 32), off, ad, y)):
        assert calls.adapter_add(*args, 36, 4096, 0) == -1
    assert calls.adapter_add(y) == -1 and calls.norm_residual() == -1
    assert not got
