"""Host-side checks of the attention half's calls (no GPU): every refusal is made before any device is touched, with its
status and, for the Python binding, its exception."""
import ctypes

import pytest

OK, INVALID, SHAPE, WS_SMALL, MISALIGNED, NO_DEVICE = 0, 1, 2, 3, 4, 7
MB = 1 << 20


@pytest.fixture(scope="module")
def m():
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    import nvfp4_w4a4_mixture_gb300 as m

    m.lib()
    return m


@pytest.fixture
def no_gpu():
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses that pass every check: only where nothing can be launched")


def p(addr):
    return None if addr is None else ctypes.c_void_p(addr)


def cache(m, dtype=0, n_pages=8, page=16, n_kv=2, D=128, k=100 * MB, v=120 * MB, ld=None, ks=None, vs=None):
    ld = ld or (page * n_kv * D, n_kv * D, D)
    return m.KvCacheDesc(dtype, n_pages, page, n_kv, D, k, v, *ld, ks, vs)


def requests(m, S=2, max_pages=4, off=200 * MB, lens=201 * MB, pages=202 * MB, ld=4):
    return m.RequestsDesc(S, max_pages, off, lens, pages, ld)


def append(m, C=None, R=None, n_q=4, rot=64, inv=210 * MB, w_q=211 * MB, w_k=212 * MB, eps=1e-6, q=MB, ld_q=512, k=2 * MB,
           ld_k=256, v=3 * MB, ld_v=256, T=4, out=4 * MB, ld_o=512, ws=300 * MB, nbytes=4096):
    d = m.RotaryDesc(n_q, rot, 0, inv, w_q, w_k, eps, 0.0)
    return m.lib().moe_cache_append(ctypes.byref(C or cache(m)), ctypes.byref(R or requests(m)), ctypes.byref(d), p(q), ld_q, p(k), ld_k,
                                    p(v), ld_v, T, p(out), ld_o, p(ws), nbytes, None)


def attend(m, C=None, R=None, n_q=4, max_new=1, window=0, scale=0.1, q=MB, ld_q=512, T=4, out=4 * MB, ld_o=512, lse=None,
           ws=300 * MB, nbytes=1 << 30):
    d = m.AttentionDesc(n_q, max_new, window, scale)
    return m.lib().moe_paged_attention(ctypes.byref(C or cache(m)), ctypes.byref(R or requests(m)), ctypes.byref(d), p(q), ld_q, T, p(out),
                                       ld_o, p(lse), p(ws), nbytes, None)


@pytest.mark.parametrize("call", [append, attend])
def test_cache_and_request_refusals(m, call):
    for kw in (dict(D=96), dict(D=0), dict(n_kv=0), dict(n_kv=1025), dict(page=0), dict(page=24), dict(page=131072), dict(n_pages=0)):
        assert call(m, C=cache(m, **kw)) == SHAPE, kw
    assert call(m, C=cache(m, dtype=1)) == INVALID
    assert call(m, C=cache(m, ks=400 * MB)) == INVALID  # a scale of a bf16 cache
    assert call(m, C=cache(m, k=None)) == INVALID
    assert call(m, C=cache(m, k=100 * MB + 8)) == MISALIGNED
    assert call(m, C=cache(m, ld=(4096, 256, 132))) == MISALIGNED
    assert call(m, C=cache(m, dtype=2, ld=(4096, 264, 128))) == MISALIGNED
    assert call(m, C=cache(m, ld=(4096, 128, 128))) == INVALID   # heads on one another
    assert call(m, C=cache(m, ld=(256, 256, 128))) == INVALID    # pages on one another
    assert call(m, C=cache(m, ld=(-4096, 256, 128))) == INVALID
    assert call(m, C=cache(m, dtype=2, ks=400 * MB + 2)) == MISALIGNED
    assert call(m, R=requests(m, S=0)) == INVALID
    assert call(m, R=requests(m, max_pages=0)) == INVALID
    assert call(m, R=requests(m, off=None)) == INVALID
    assert call(m, R=requests(m, ld=3)) == INVALID
    assert call(m, R=requests(m, lens=201 * MB + 2)) == MISALIGNED
    assert call(m, T=-1) == SHAPE
    assert call(m, ws=None) == INVALID
    assert call(m, ws=300 * MB + 64) == MISALIGNED
    assert call(m, nbytes=128) == WS_SMALL


def test_append_refusals(m):
    null = ctypes.POINTER(m.KvCacheDesc)()
    assert m.lib().moe_cache_append(null, None, None, None, 0, None, 0, None, 0, 4, None, 0, None, 0, None) == INVALID
    for rot in (-16, 8, 144, 24):
        assert append(m, rot=rot) == SHAPE
    assert append(m, n_q=-1) == SHAPE
    assert append(m, eps=-1.0) == INVALID and append(m, eps=float("nan")) == INVALID
    assert append(m, rot=0) == INVALID and append(m, inv=None) == INVALID  # one without the other
    assert append(m, q=None) == INVALID and append(m, out=None) == INVALID and append(m, n_q=0) == INVALID
    assert append(m, n_q=0, q=None, out=None) == INVALID  # w_q without q
    assert append(m, k=None) == INVALID and append(m, v=None) == INVALID
    assert append(m, ld_q=504) == INVALID and append(m, ld_k=248) == INVALID
    assert append(m, ld_q=516) == MISALIGNED and append(m, v=3 * MB + 8) == MISALIGNED and append(m, w_k=212 * MB + 8) == MISALIGNED
    assert append(m, out=MB, ld_o=1024) == INVALID      # q's address with another stride
    assert append(m, out=MB + 1024) == INVALID          # a row into q
    assert append(m, out=2 * MB) == INVALID and append(m, out=100 * MB) == INVALID and append(m, out=202 * MB) == INVALID
    assert append(m, k=100 * MB) == INVALID             # keys inside the cache
    assert append(m, C=cache(m, v=100 * MB)) == INVALID


def test_attention_refusals(m):
    for kw in (dict(n_q=0), dict(n_q=3), dict(n_q=130), dict(max_new=0), dict(max_new=17)):
        assert attend(m, **kw) == SHAPE, kw
    assert attend(m, window=-1) == INVALID
    assert attend(m, scale=float("nan")) == INVALID and attend(m, scale=float("inf")) == INVALID
    assert attend(m, q=None) == INVALID and attend(m, out=None) == INVALID
    assert attend(m, ld_q=504) == INVALID and attend(m, out=4 * MB + 8) == MISALIGNED and attend(m, lse=5 * MB + 2) == MISALIGNED
    assert attend(m, out=MB + 1024) == INVALID and attend(m, out=MB, ld_o=1024) == INVALID
    assert attend(m, out=101 * MB - MB) == INVALID      # on the cache
    assert attend(m, lse=MB) == INVALID and attend(m, lse=4 * MB) == INVALID and attend(m, lse=201 * MB) == INVALID
    assert attend(m, T=1 << 30) == SHAPE  # 2^32 rows of heads


def test_workspace_bytes(m):
    f = m.moe_attention_workspace_bytes
    assert f(1, 3, 2, 128, 1) == 0 and f(1, 2, 2, 96, 1) == 0 and f(-1, 2, 2, 128, 1) == 0 and f(1, 2, 2, 128, 17) == 0
    assert 0 < f(1, 16, 2, 128, 1) < f(1, 16, 2, 256, 1) < f(1, 16, 2, 256, 16)
    assert f(100000, 16, 2, 128, 1) >= f(1, 16, 2, 128, 1) + 8 * 99999


def test_accepts(m, no_gpu):
    assert append(m) == NO_DEVICE
    assert append(m, out=MB) == NO_DEVICE
    assert append(m, n_q=0, q=None, out=None, w_q=None) == NO_DEVICE
    assert append(m, rot=0, inv=None, w_q=None, w_k=None) == NO_DEVICE
    # columns of one buffer of 1024 elements a row
    assert append(m, q=MB, ld_q=1024, k=MB + 1024, ld_k=1024, v=MB + 1536, ld_v=1024) == NO_DEVICE
    assert attend(m) == NO_DEVICE
    assert attend(m, out=MB) == NO_DEVICE
    assert attend(m, C=cache(m, ld=(4096, 128, 2048))) == NO_DEVICE                       # heads first
    assert attend(m, C=cache(m, k=100 * MB, v=100 * MB + 8192, ld=(8192, 256, 128))) == NO_DEVICE  # keys and values by turns


def quant(m, x=MB, ld=2048, T=4, K=2048, codes=2 * MB, scale=3 * MB):
    return m.lib().moe_quantize_fp8(p(x), ld, T, K, p(codes), p(scale), None)


def gemm(m, a=MB, sa=2 * MB, b=10 * MB, sb=3 * MB, T=4, N=512, K=2048, out=4 * MB, dt=0, ld=512, ws=300 * MB, nbytes=4096):
    return m.lib().moe_gemm_fp8(p(a), p(sa), p(b), p(sb), T, N, K, p(out), dt, ld, p(ws), nbytes, None)


def test_overlap_of_more_than_two_gigabytes_of_scales(m):
    """600,000,000 rows: an output over the last of their scales."""
    T, G = 600_000_000, 1 << 40
    kw = dict(T=T, K=16, N=8, ld=8, a=G, b=2 * G, sb=3 * G, sa=4 * G)
    assert gemm(m, out=4 * G + 4 * T - 16, ws=None, **kw) == INVALID and b"overlaps" in m.lib().moe_last_error_detail()
    assert gemm(m, out=4 * G + 4 * T, ws=None, **kw) == INVALID and b"overlaps" not in m.lib().moe_last_error_detail()


def test_fp8_refusals(m):
    for K in (0, 8, 24, -16, 65552):
        assert quant(m, K=K) == SHAPE and gemm(m, K=K) == SHAPE
    assert quant(m, T=-1) == SHAPE and gemm(m, T=-1) == SHAPE
    assert quant(m, x=None) == INVALID and quant(m, codes=None) == INVALID and quant(m, scale=None) == INVALID
    assert quant(m, ld=2040) == INVALID and quant(m, ld=2052) == MISALIGNED and quant(m, codes=2 * MB + 8) == MISALIGNED
    assert quant(m, codes=MB) == INVALID and quant(m, scale=MB) == INVALID and quant(m, scale=2 * MB) == INVALID
    for N in (0, 4, 12, 1 << 21):
        assert gemm(m, N=N) == SHAPE
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(dt=2), dict(dt=-1), dict(ld=504), dict(ws=None)):
        assert gemm(m, **kw) == INVALID, kw
    for kw in (dict(a=MB + 8), dict(b=10 * MB + 8), dict(sa=2 * MB + 2), dict(out=4 * MB + 8), dict(ld=516), dict(ws=300 * MB + 16)):
        assert gemm(m, **kw) == MISALIGNED, kw
    for out in (MB, 2 * MB, 3 * MB, 10 * MB + 4096):
        assert gemm(m, out=out) == INVALID
    assert gemm(m, nbytes=128) == WS_SMALL


def test_empty_batches(m):
    assert append(m, T=0, q=None, k=None, v=None, out=None, ws=None) == OK
    assert attend(m, T=0, q=None, out=None, ws=None) == OK
    assert quant(m, T=0, x=None, codes=None, scale=None) == OK and gemm(m, T=0, a=None, out=None, ws=None) == OK
    assert append(m, T=0, rot=8) == SHAPE and attend(m, T=0, n_q=3) == SHAPE and quant(m, T=0, K=8) == SHAPE and gemm(m, T=0, N=12) == SHAPE


def test_python_refusals(m):
    import torch

    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    c = torch.zeros(5, 16, 2, 64, dtype=bf)
    off, lens, pages = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1, 2, dtype=i32)
    with pytest.raises(TypeError, match="k must be a CUDA tensor"):
        m.moe_cache_append(q, k, k, c, c, off, lens, pages)
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        m.moe_paged_attention(q, c, c, off, lens, pages)
    with pytest.raises(ValueError, match="k_cache of"):
        m.moe_paged_attention(q, torch.zeros(5, 16, 2, 128, dtype=bf), c, off, lens, pages)
    with pytest.raises(TypeError, match="x must be a CUDA tensor"):
        m.moe_quantize_fp8(torch.zeros(2, 128, dtype=bf))
    z = torch.zeros(2, 128).to(torch.float8_e4m3fn)
    with pytest.raises(TypeError, match="CUDA tensor"):
        m.moe_gemm_fp8(z, torch.zeros(2, 1), z, torch.zeros(1, 1))
