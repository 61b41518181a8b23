"""GPU: the operators around the expert layer against plain implementations in 64 bits.

Tolerances, from the kernels' arithmetic (u = 2^-24, half a step of FP32; h = 2^-8, of bf16):
  norms    a row's sum of squares passes through at most 128 roundings (64 of them after the square root),
           the other steps through 12: 80 u relative to |alpha r| + |g u|; a bf16 output adds h of its value
  weights  a score is off by 8 u (exponential, sum, division), the softmax's and the weights' sums by at most 40 u
           each, the last steps by 4: 96 u
  adapters A x is summed in FP32 over K terms (K u of the sum of magnitudes) and then held in 16 bits or
           more (2^-16); the output is rounded to bf16 (h)
Expert ids have to be equal.
"""
import itertools

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, HALF_BF16 = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import nvfp4_w4a4_mixture_gb300 as m
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    m.lib()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def strided(t, pad):
    """The same values in rows `pad` elements further apart."""
    if t is None or pad == 0:
        return t
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    buf[:, : t.shape[1]] = t
    return buf[:, : t.shape[1]]


# ------------------------------------------------------------------------------------------------
# norms
# ------------------------------------------------------------------------------------------------
def norm_ref(y, r, w_post, w_pre, gate, alpha, eps, off):
    """(r', its magnitude |alpha r| + |g u|, 1 / rms of r' times the weight) in 64 bits."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    y, r, w_post, w_pre, gate = map(d, (y, r, w_post, w_pre, gate))
    T, H = (y if y is not None else r).shape
    total, size = torch.zeros(T, H, dtype=torch.float64, device="cuda"), 0.0
    if r is not None:
        total = total + alpha * r
        size = size + (alpha * r).abs()
    if y is not None:
        u = y
        if w_post is not None:
            u = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * (off + w_post)
        if gate is not None:
            u = gate * u
        total = total + u
        size = size + u.abs()
    f = None if w_pre is None else (off + w_pre) / torch.sqrt((total * total).mean(1, keepdim=True) + eps)
    return total, size, f


def check_norm(moe, T, H, rt=BF, gate=None, gate_type=BF, post=True, pre=True, with_y=True, with_r=True, alpha=1.0, off=0.0,
               eps=1e-6, pad=0, in_place=False, seed=0):
    g = gen(seed * 100003 + T * 131 + H)
    y = strided(randn(g, T, H, std=0.5, dtype=BF), pad) if with_y else None
    r = strided(randn(g, T, H, std=2.0, dtype=rt), pad) if with_r else None
    w_post = randn(g, H, std=0.1, mean=1 - off, dtype=BF) if post else None
    w_pre = randn(g, H, std=0.1, mean=1 - off, dtype=BF) if pre else None
    shape = {None: None, "channel": (H,), "token": (T, 1), "element": (T, H), "one": (1, 1)}[gate]
    gt = None if shape is None else randn(g, *shape, dtype=gate_type)
    if gate == "element":
        gt = strided(gt, pad)
    ref, size, f = norm_ref(y, r, w_post, w_pre, gt, alpha, eps, off)
    r_out = x_out = None
    if in_place:
        r_out, x_out = r, y
    elif pad:
        r_out = strided(torch.empty(T, H, dtype=rt if with_r else BF, device="cuda"), 2 * pad)
        x_out = strided(torch.empty(T, H, dtype=BF, device="cuda"), pad) if pre else None
    got_r, got_x = moe.moe_norm_residual(y, r, w_post=w_post, w_pre=w_pre, gate=gt, residual_scale=alpha, eps=eps, w_offset=off,
                                         out=(r_out, x_out))
    torch.cuda.synchronize()
    if r_out is not None:
        assert got_r is r_out
    half = HALF_BF16 if got_r.dtype == BF else U
    err = (got_r.double() - ref).abs()
    assert torch.all(err <= half * ref.abs() + 80 * U * size), float((err / (size + 1e-30)).max())
    if not pre:
        assert got_x is None
        return
    xr = ref * f
    err = (got_x.double() - xr).abs()
    assert torch.all(err <= HALF_BF16 * xr.abs() + 80 * U * f.abs() * (size + ref.abs())), float(err.max())


@pytest.mark.parametrize("T,H", [(1, 8), (1, 2048), (4, 2048), (3, 24), (33, 136), (7, 1032), (5, 2056), (9, 4096), (70, 8192),
                                 (2, 8184), (300, 2048), (1000, 512), (4097, 256), (2500, 2056),
                                 (2000, 768), (701, 640), (1999, 1024), (1501, 1272), (1500, 1536), (901, 2824), (900, 4096),
                                 (700, 4608), (500, 5128), (305, 6152), (613, 8192)])
def test_norm_sizes(moe, T, H):
    check_norm(moe, T, H)
    check_norm(moe, T, H, rt=torch.float32, gate="channel", alpha=0.5, off=1.0, seed=1)


@pytest.mark.parametrize("gate,gate_type", list(itertools.product(["channel", "token", "element", "one"], [BF, torch.float32])))
def test_norm_gates(moe, gate, gate_type):
    for T, H in ((5, 2048), (130, 264)):
        check_norm(moe, T, H, gate=gate, gate_type=gate_type, alpha=0.7071)
        check_norm(moe, T, H, gate=gate, gate_type=gate_type, post=False, rt=torch.float32, pad=8)


@pytest.mark.parametrize("kw", [dict(with_y=False, post=False), dict(with_r=False), dict(pre=False), dict(post=False, pre=False),
                                dict(pad=8), dict(pad=24, rt=torch.float32), dict(in_place=True),
                                dict(in_place=True, pad=16, gate="element"), dict(eps=0.0), dict(eps=0.5, off=1.0)])
def test_norm_forms(moe, kw):
    for T, H in ((1, 2048), (6, 2048), (259, 1048), (20, 8192)):
        check_norm(moe, T, H, **kw)


def test_norm_rows_of_zeros_and_no_numbers(moe):
    # a row of zeros is divided by sqrt(eps); a row with an infinity or NaN is the formula's, and no other row's matter
    g = gen(5)
    for T, H in ((8, 2048), (2000, 264)):
        y, r = randn(g, T, H, dtype=BF), randn(g, T, H, dtype=BF)
        w = randn(g, H, mean=1.0, std=0.1, dtype=BF)
        clean = moe.moe_norm_residual(y, r, w_post=w, w_pre=w)
        y[1], r[1] = 0.0, 0.0
        y[3, 7] = float("inf")
        r[5, H - 1] = float("nan")
        r_out, x_out = moe.moe_norm_residual(y, r, w_post=w, w_pre=w)
        assert torch.all(r_out[1] == 0) and torch.all(x_out[1] == 0)
        # 1 / rms is 0 there: inf * 0 at the infinity, the residual alone elsewhere
        assert bool(r_out[3, 7].isnan()) and torch.equal(r_out[3, :7], r[3, :7]) and torch.all(x_out[3].isnan())
        assert bool(r_out[5, H - 1].isnan()) and not bool(r_out[5, : H - 1].isnan().any()) and torch.all(x_out[5].isnan())
        rest = [i for i in range(T) if i not in (1, 3, 5)]
        assert torch.equal(r_out[rest], clean[0][rest]) and torch.equal(x_out[rest], clean[1][rest])


# ------------------------------------------------------------------------------------------------
# expert selection
# ------------------------------------------------------------------------------------------------
def select_ref(l, k, bias, score, G, keep, top2, renorm, scale):
    """(ids, weights) in 64 bits by sorting, the masked experts after the others."""
    T, E = l.shape
    l = l.astype(np.float64)
    real = l > -np.inf  # neither -inf nor NaN
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = np.where(real, 1 / (1 + np.exp(-l)), 0.0)
        else:
            m = np.where(real, l, -np.inf).max(1, keepdims=True)
            s = np.where(real, np.where(l == m, 1.0, np.exp(l - m)), 0.0)
            s = np.where(real, s / s.sum(1, keepdims=True), 0.0)
        # without a bias a larger logit has a larger score, also where 64 bits no longer tell them apart
        c = s + bias.astype(np.float64) if bias is not None else np.where(real, l, -np.inf)
        real = real & (c > -np.inf)
        c = np.where(real, c, -np.inf)
        v = np.where(real, s if bias is None and top2 else c, -np.inf).reshape(T, G, E // G)
        top = -np.sort(-v, axis=2)
        gv = top[:, :, 0]
        if top2 and E // G > 1:
            gv = np.where(top[:, :, 1] > -np.inf, gv + top[:, :, 1], gv)
    ids, w = np.empty((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        stay = np.zeros(G, bool)
        stay[np.lexsort((np.arange(G), -gv[t]))[:keep]] = True
        e = np.flatnonzero(np.repeat(stay, E // G))
        order = e[np.lexsort((e, -c[t, e], ~real[t, e]))][:k]
        ids[t] = order
        w[t] = np.where(real[t, order], s[t, order], 0.0)
        total = w[t].sum()
        if renorm:
            w[t] = w[t] / total if total > 0 else 0.0
    return ids, w * scale


def check_select(moe, logits, k, bias=None, score="sigmoid", G=1, keep=1, top2=True, renorm=True, scale=1.0):
    ids, w = moe.moe_select_experts(logits, k, bias=bias, score=moe.SCORE_SIGMOID if score == "sigmoid" else moe.SCORE_SOFTMAX,
                                    n_group=G, topk_group=keep, group_score=moe.GROUP_TOP2 if top2 else moe.GROUP_MAX,
                                    renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    ref_ids, ref_w = select_ref(logits.float().cpu().numpy(), k, None if bias is None else bias.cpu().numpy(), score, G, keep,
                                top2, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    err = np.abs(w.double().cpu().numpy() - ref_w)
    assert np.all(err <= 96 * U * np.abs(ref_w) + 1e-37), float((err / (np.abs(ref_w) + 1e-37)).max())


@pytest.mark.parametrize("T,E,k,G,keep", [
    (1, 1, 1, 1, 1), (1, 512, 10, 1, 1), (4, 512, 10, 1, 1), (3, 5, 5, 1, 1), (33, 60, 4, 1, 1), (70, 16, 2, 1, 1),
    (17, 1024, 32, 1, 1), (5, 1024, 32, 32, 16), (100, 256, 8, 8, 4), (65, 160, 6, 8, 3), (9, 96, 12, 32, 4), (50, 31, 7, 1, 1),
    (40, 7, 3, 7, 3), (1000, 512, 10, 8, 4), (2049, 384, 16, 2, 1), (3, 33, 32, 3, 3), (11, 640, 9, 5, 2), (6, 1023, 17, 3, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_sizes(moe, T, E, k, G, keep, score):
    g = gen(T * 7 + E)
    bias = randn(g, E, std=0.02)
    for dtype, b, top2, renorm, scale in ((torch.float32, bias, True, True, 1.0), (torch.float32, None, False, False, 2.5),
                                          (BF, None, True, True, 1.0), (BF, bias, False, True, 2.5)):
        check_select(moe, randn(g, T, E, dtype=dtype), k, bias=b, score=score, G=G, keep=keep, top2=top2, renorm=renorm, scale=scale)


@pytest.mark.parametrize("T,E,k,G,keep", [(2433, 16, 2, 1, 1), (2600, 60, 4, 1, 1), (2432, 128, 8, 8, 4), (3001, 160, 6, 8, 3),
                                          (2501, 192, 12, 16, 8), (2700, 256, 8, 8, 4), (2435, 31, 7, 1, 1), (2433, 250, 10, 5, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_select_many_tokens(moe, T, E, k, G, keep, score):
    # two tokens a warp; an odd number of them, rows of equal, masked and nearly equal values among the others
    g = gen(T + E)
    bias = randn(g, E, std=0.02)
    level = (0.75 - torch.sigmoid(torch.linspace(-1, 1, E, device="cuda").double())).float()
    for dtype, b, top2, renorm in ((torch.float32, bias, True, True), (torch.float32, None, False, False), (BF, None, True, True),
                                   (BF, bias, False, True), (torch.float32, level, True, True)):
        l = randn(g, T, E, dtype=dtype)
        l[5], l[8] = 0.25, float("-inf")
        l[11, ::2], l[14, 1::2] = float("-inf"), float("nan")
        l[17, : E // 2], l[20, 3] = float("-inf"), float("inf")
        l[100:140] = torch.linspace(-1, 1, E, device="cuda")
        l[T - 1] = 1.0
        check_select(moe, l, k, bias=b, score=score, G=G, keep=keep, top2=top2, renorm=renorm)


def test_select_strided_and_unaligned_rows(moe):
    g = gen(3)
    for E, pad in ((512, 1), (512, 16), (160, 3), (256, 8)):
        for dtype in (torch.float32, BF):
            l = strided(randn(g, 37, E, dtype=dtype), pad)
            check_select(moe, l, 8, bias=randn(g, E, std=0.02), G=8, keep=4)
            flat = torch.empty(37 * (E + pad) + 1, dtype=dtype, device="cuda").fill_(float("nan"))
            view = flat[1:].view(37, E + pad)[:, :E]  # a base on an element's alignment alone
            view.copy_(l)
            check_select(moe, view, 8, bias=randn(g, E, std=0.02), score="softmax")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (8, 3)])
def test_select_ties(moe, score, G, keep):
    # equal logits: the lowest ids and groups; two values only, and rows of one value
    g = gen(11)
    E = 512
    l = (torch.rand(64, E, generator=g, device="cuda") < 0.3).float()
    l[0], l[1] = 0.0, -3.0
    for bias in (None, torch.zeros(E, device="cuda"), (torch.arange(E, device="cuda") % 3) * 0.25):
        check_select(moe, l, 10, bias=bias, score=score, G=G, keep=keep)
        check_select(moe, l.to(BF), 10, bias=bias, score=score, G=G, keep=keep, top2=False)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,keep", [(1, 1), (8, 4)])
def test_select_values_nearer_than_32_bits_tell(moe, score, G, keep):
    # a bias that levels the scores: every choice value of the first token lies within a few units of the last place of one number
    g = gen(12)
    E = 256
    l = randn(g, 40, E)
    s = torch.sigmoid(l[0].double()) if score == "sigmoid" else torch.softmax(l[0].double(), 0)
    bias = (0.75 - s).float()
    check_select(moe, l, 8, bias=bias, score=score, G=G, keep=keep)
    check_select(moe, l[:1].repeat(300, 1) + torch.arange(300, device="cuda")[:, None] * 1e-7, 8, bias=bias, score=score, G=G, keep=keep)
    # logits one unit of the last place apart, in an order that does not follow the ids
    near = torch.nextafter(torch.ones(E, device="cuda"), torch.full((E,), 2.0, device="cuda"))
    pick = torch.randint(0, 2, (40, E), generator=g, device="cuda").bool()
    check_select(moe, torch.where(pick, near, torch.ones(E, device="cuda")), 8, score=score, G=G, keep=keep)
    check_select(moe, torch.where(pick, near, torch.ones(E, device="cuda")), 8, bias=torch.full((E,), 0.5, device="cuda"),
                 score=score, G=G, keep=keep)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_select_masked_logits(moe, score, with_bias):
    g = gen(13)
    E, k, inf, nan, low = 64, 8, float("inf"), float("nan"), torch.finfo(torch.float32).min
    l = randn(g, 16, E)
    l[0] = -inf                      # nothing left: the lowest ids, weights 0
    l[1] = nan
    l[2] = -inf
    l[2, 50] = 0.3                   # one expert left
    l[3, ::2] = -inf
    l[4, 1::3] = nan
    l[5] = low                       # a mask of the type's lowest value is a number like another
    l[5, 40:43] = 1.0
    l[6, 7], l[6, 60] = inf, inf
    l[7] = inf
    l[8, :32] = -inf                 # whole groups masked
    l[9, 8:] = -inf                  # fewer left than chosen
    l[10] = l[10] * 30.0             # scores that underflow
    l[11] = -200.0
    l[11, 5] = -100.0
    bias = randn(g, E, std=0.02) if with_bias else None
    for G, keep in ((1, 1), (8, 2), (16, 4)):
        for top2 in (False, True):
            check_select(moe, l, k, bias=bias, score=score, G=G, keep=keep, top2=top2)
    if with_bias:
        b = bias.clone()
        b[3], b[4], b[5], b[20] = -inf, nan, inf, inf
        for G, keep in ((1, 1), (8, 2)):
            check_select(moe, l, k, bias=b, score=score, G=G, keep=keep)
    check_select(moe, l.to(BF)[:5], k, bias=bias, score=score)


def test_select_agrees_with_the_layers_router(moe):
    # softmax, renormalised, without groups: what moe_route_topk chooses, from the logits that it returns
    from nvfp4_w4a4_mixture_gb300 import workloads as wl

    H, E, k = 256, 64, 6
    w_r = torch.from_numpy(wl.gen_router(0, E, H)).to(BF).cuda()
    dummy = (torch.zeros(1, 1, 8, dtype=torch.uint8, device="cuda"),) * 2 + (torch.ones(1, 2, device="cuda"),)
    layer = moe.MoeLayer(H, E, k, 128, w_r, dummy, dummy, torch.ones(E + 1, device="cuda"), prepacked=True)
    x = torch.from_numpy(wl.gen_x(1, 200, H)).to(BF).cuda()
    ids, w, _, logits = moe.moe_route_topk(x, layer, want_logits=True)
    got_ids, got_w = moe.moe_select_experts(logits, k)
    assert torch.equal(ids, got_ids)
    assert float((w - got_w).abs().max()) <= 1e-6


# ------------------------------------------------------------------------------------------------
# adapters
# ------------------------------------------------------------------------------------------------
def adapter_case(lens, adapters, n, r, K, N, seed=0, pad=0):
    g = gen(seed * 7 + sum(lens) + r)
    T = sum(lens)
    off = torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32, device="cuda")
    return dict(x=strided(randn(g, T, K, dtype=BF), pad), y=strided(randn(g, T, N, std=0.5, dtype=BF), pad),
                a=randn(g, n, r, K, std=0.02, dtype=BF), b=randn(g, n, N, r, std=0.05, dtype=BF), scale=randn(g, n, std=0.3, mean=2.0),
                seg_offsets=off, seg_adapter=torch.tensor(adapters, dtype=torch.int32, device="cuda"))


def check_adapter(moe, c, out=None, skip=()):
    y = c["y"].clone()
    K = c["x"].shape[1]
    got = moe.moe_adapter_add(**c, out=out)
    moe.moe_read_device_status()
    off = c["seg_offsets"].tolist()
    for s, ad in enumerate(c["seg_adapter"].tolist()):
        rows = slice(off[s], off[s + 1])
        if s in skip or off[s] == off[s + 1]:
            continue
        if ad < 0:
            assert torch.equal(got[rows], y[rows])
            continue
        x, a, b, f = c["x"][rows].double(), c["a"][ad].double(), c["b"][ad].double(), float(c["scale"][ad])
        h = x @ a.T
        ref = y[rows].double() + f * (h @ b.T)
        h_err = 2.0 ** -16 * h.abs() + K * U * (x.abs() @ a.abs().T)
        # the terms' own rounding and their FP32 sum over the rank
        slack = abs(f) * ((h_err + (a.shape[0] + 4) * U * h.abs()) @ b.abs().T) + 2 * U * ref.abs()
        err = (got[rows].double() - ref).abs()
        assert torch.all(err <= HALF_BF16 * ref.abs() + slack), (s, float((err - HALF_BF16 * ref.abs()).max()))
        assert float((got[rows].double() - ref).norm()) <= HALF_BF16 * float(ref.norm())
    return got


@pytest.mark.parametrize("lens,adapters", [
    ([1], [0]), ([4], [1]), ([1, 1, 1, 1], [2, 0, -1, 2]), ([3, 1], [0, 1]), ([0, 5, 0, 0, 2, 0], [0, 1, 2, -1, 2, 0]),
    ([127], [0]), ([128], [1]), ([129], [2]), ([257, 1, 130], [0, 2, 1]), ([40], [-1]), ([9, 8, 7, 33, 31, 32, 65], [0, 1, 2, 0, -1, 2, 1])])
@pytest.mark.parametrize("r,K,N", [(8, 64, 64), (16, 2048, 2048), (40, 264, 520)])
def test_adapter_segments(moe, lens, adapters, r, K, N):
    check_adapter(moe, adapter_case(lens, adapters, 3, r, K, N))


@pytest.mark.parametrize("r,K,N", [(8, 8, 8), (16, 16, 24), (24, 72, 56), (32, 128, 128), (48, 2056, 1032), (56, 200, 2000), (64, 2048, 2048),
                                   (96, 512, 264), (128, 2048, 2048), (128, 8192, 136), (8, 136, 8192), (120, 1000, 8)])
def test_adapter_shapes(moe, r, K, N):
    check_adapter(moe, adapter_case([150, 3, 1, 17], [1, 0, -1, 1], 2, r, K, N))


@pytest.mark.parametrize("r,K,N", [(8, 8, 8), (16, 72, 56), (24, 200, 2000), (48, 2056, 1032), (64, 512, 264), (120, 1000, 8), (128, 2048, 2048)])
@pytest.mark.parametrize("lens", [[1100], [1500, 3, 1, 900, 128, 700], [129, 2] * 100, [64, 65, 1, 40, 63, 8, 128, 9, 100, 33] * 9,
                                  [700] * 8 + [1, 7, 31] * 6])
def test_adapter_long_requests(moe, r, K, N, lens):
    # enough rows for the kernel of 128-row tiles, one CTA a tile or several
    check_adapter(moe, adapter_case(lens, [(i % 4) - 1 if i else 1 for i in range(len(lens))], 3, r, K, N))


def test_adapter_many_requests(moe):
    rng = np.random.default_rng(0)
    lens = [int(v) for v in rng.integers(0, 6, 700)]
    check_adapter(moe, adapter_case(lens, [int(v) for v in rng.integers(-1, 20, 700)], 20, 16, 256, 256))
    lens = [int(v) for v in rng.integers(1, 400, 30)]
    check_adapter(moe, adapter_case(lens, [int(v) for v in rng.integers(-1, 5, 30)], 5, 64, 512, 384))
    check_adapter(moe, adapter_case([5000], [1], 2, 32, 2048, 2048))


@pytest.mark.parametrize("lens", [[1] * 400, [40, 1, 33] * 60, [130, 2] * 150])
def test_adapter_tiles_with_and_without_adapter_in_turn(moe, lens):
    # several tiles a multiprocessor, many slices each, copied tiles between the others
    check_adapter(moe, adapter_case(lens, [(i % 5) - 1 if i % 3 else -1 for i in range(len(lens))], 4, 24, 1032, 2048))


@pytest.mark.parametrize("lens,r,K,N", [([1500, 3, 1, 900, 128, 700], 128, 2048, 2048), ([700] * 20, 64, 1032, 2056),
                                        ([129, 2] * 150, 32, 2048, 2048), ([1] * 256, 16, 2048, 2048), ([3, 1, 5], 64, 2048, 2048),
                                        ([130, 60, 33, 1, 77] * 16, 40, 2056, 1032)])
def test_adapter_repeats_itself(moe, lens, r, K, N):
    # the same bits every time, also while other work keeps the memory busy
    c = adapter_case(lens, [(i % 4) - 1 if i else 1 for i in range(len(lens))], 3, r, K, N)
    want = check_adapter(moe, c).clone()
    out, busy = torch.empty_like(want), randn(gen(1), 2048, 2048)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(300):
        out.fill_(7.0)
        if i % 3 == 1:
            busy = busy @ busy * 1e-3
        moe.moe_adapter_add(**c, out=out)
        same &= (out == want).all()
    moe.moe_read_device_status()
    assert bool(same)


def test_adapter_strides_and_in_place(moe):
    for lens in ([5, 1], [300, 70]):
        c = adapter_case(lens, [1, 0], 2, 16, 264, 136, pad=24)
        want = check_adapter(moe, c)
        into = strided(torch.zeros_like(want), 40)
        assert check_adapter(moe, c, out=into) is into and torch.equal(into, want)
        assert torch.equal(check_adapter(moe, c, out=c["y"]), want)
        bare = adapter_case(lens, [-1, -1], 2, 16, 264, 136)
        y = bare["y"].clone()
        assert torch.equal(check_adapter(moe, bare, out=bare["y"]), y)


def test_adapter_rows_with_no_numbers_stay_alone(moe):
    # a row's infinity or NaN reaches no other row
    for lens in ([6, 3], [140, 30]):
        c = adapter_case(lens, [0, 1], 2, 16, 256, 256)
        clean = check_adapter(moe, c)
        c["x"][2, 5] = float("nan")
        c["x"][lens[0] + 1, 9] = float("inf")
        got = moe.moe_adapter_add(**c)
        rest = [i for i in range(sum(lens)) if i not in (2, lens[0] + 1)]
        assert torch.equal(got[rest], clean[rest])
        assert torch.all(got[2].isnan()) and not bool(got[lens[0] + 1].isfinite().any())


def test_adapter_reports_bad_segments(moe):
    # adapters out of range: their rows are not written, the others' are right, the status says so and is cleared
    for lens in ([3, 2, 4], [200, 10, 150]):
        c = adapter_case(lens, [0, 2, 1], 2, 16, 256, 256)
        for bad in (2, -2, 1 << 30):
            c["seg_adapter"][1] = bad
            out = torch.full_like(c["y"], 7.0)
            moe.moe_adapter_add(**c, out=out)
            with pytest.raises(moe.MoeError, match="INVALID_ARG"):
                moe.moe_read_device_status()
            moe.moe_read_device_status()
            assert torch.all(out[lens[0]: lens[0] + lens[1]] == 7.0)
            c["seg_adapter"][1] = 0
            want = check_adapter(moe, c)
            keep = list(range(lens[0])) + list(range(lens[0] + lens[1], sum(lens)))
            assert torch.equal(out[keep], want[keep])
        for off in ([0, 3, 5, sum(lens) + 1], [0, 3, 5, sum(lens) - 1], [1, 3, 5, sum(lens)], [0, -3, 5, sum(lens)],
                    [0, 5, 3, sum(lens)], [0, 1 << 30, 5, sum(lens)], [-(1 << 31), 3, 5, sum(lens)], [0, 3, 5, (1 << 31) - 1]):
            c["seg_offsets"].copy_(torch.tensor(off, dtype=torch.int32))
            moe.moe_adapter_add(**c)
            with pytest.raises(moe.MoeError, match="INVALID_ARG"):
                moe.moe_read_device_status()


# ------------------------------------------------------------------------------------------------
# all of them: repeatable, on other streams, in a graph
# ------------------------------------------------------------------------------------------------
def calls(moe, T):
    g = gen(T)
    y, r = randn(g, T, 2048, dtype=BF), randn(g, T, 2048, dtype=BF)
    w = randn(g, 2048, std=0.1, mean=1.0, dtype=BF)
    l, bias = randn(g, T, 512), randn(g, 512, std=0.02)
    c = adapter_case([T // 2, T - T // 2], [1, 0], 2, 16, 2048, 2048)
    return [(lambda out: moe.moe_norm_residual(y, r, w_post=w, w_pre=w, out=out), (r.shape, BF), (y.shape, BF)),
            (lambda out: moe.moe_select_experts(l, 10, bias=bias, score=1, n_group=8, topk_group=4, out=out),
             ((T, 10), torch.int32), ((T, 10), torch.float32)),
            (lambda out: (moe.moe_adapter_add(**c, out=out[0]), out[0]), (c["y"].shape, BF), (c["y"].shape, BF))]


@pytest.mark.parametrize("T", [4, 300])
def test_repeatable_on_a_stream_and_in_a_graph(moe, T):
    for f, *shapes in calls(moe, T):
        new = lambda: tuple(torch.zeros(s, dtype=d, device="cuda") for s, d in shapes)  # noqa: E731
        first, again, other, graphed = new(), new(), new(), new()
        f(first)
        f(again)
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            f(other)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f(graphed)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for got in (again, other, graphed):
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("T", [1, 4, 300])
def test_both_marshallings_give_the_same(moe, monkeypatch, T):
    for f, *shapes in calls(moe, T):
        new = lambda: tuple(torch.zeros(s, dtype=d, device="cuda") for s, d in shapes)  # noqa: E731
        first, again = new(), new()
        f(first)
        monkeypatch.setattr(moe, "_calls", None)
        f(again)
        monkeypatch.undo()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refuses_on_the_device(moe):
    y = torch.zeros(4, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    with pytest.raises(TypeError, match="w_pre"):
        moe.moe_norm_residual(y, y, w_pre=w.float())
    with pytest.raises(ValueError, match="gate"):
        moe.moe_norm_residual(y, y, gate=torch.ones(3, 64, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="y must"):
        moe.moe_norm_residual(y.t().contiguous().t(), y)
    with pytest.raises(moe.MoeError, match="overlaps"):
        moe.moe_norm_residual(y, y.clone(), w_pre=w, out=(y, torch.empty_like(y)))
    with pytest.raises(moe.MoeError, match="k=5"):
        moe.moe_select_experts(torch.zeros(4, 4, device="cuda"), 5)
    with pytest.raises(TypeError, match="seg_offsets"):
        moe.moe_adapter_add(y, y, torch.zeros(1, 8, 64, dtype=BF, device="cuda"), torch.zeros(1, 64, 8, dtype=BF, device="cuda"),
                            torch.ones(1, device="cuda"), torch.tensor([0, 4], device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_outputs_stay_inside_their_rows(moe):
    # what lies between and behind the outputs' rows is left alone
    T, H = 37, 264
    g = gen(1)
    y, r, w = randn(g, T, H, dtype=BF), randn(g, T, H, dtype=BF), randn(g, H, dtype=BF)
    r_buf, x_buf, a_buf = (torch.full((T + 2, H + 16), 5.0, dtype=BF, device="cuda") for _ in range(3))
    moe.moe_norm_residual(y, r, w_pre=w, out=(r_buf[1:T + 1, :H], x_buf[1:T + 1, :H]))
    c = adapter_case([T - 1, 1], [1, 0], 2, 24, 264, H)
    moe.moe_adapter_add(**c, out=a_buf[1:T + 1, :H])
    for buf in (r_buf, x_buf, a_buf):
        assert torch.all(buf[0] == 5) and torch.all(buf[T + 1] == 5) and torch.all(buf[:, H:] == 5)
    ids, wt = torch.full((T + 2, 6), -7, dtype=torch.int32, device="cuda"), torch.full((T + 2, 6), 5.0, device="cuda")
    moe.moe_select_experts(randn(g, T, 64), 6, out=(ids[1:T + 1], wt[1:T + 1]))
    assert torch.all(ids[0] == -7) and torch.all(ids[T + 1] == -7) and torch.all(wt[0] == 5) and torch.all(wt[T + 1] == 5)
    assert torch.all(ids[1:T + 1] >= 0)


def test_empty_batches(moe):
    e = torch.empty
    y = e(0, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    r_out, x_out = moe.moe_norm_residual(y, y, w_post=w, w_pre=w)
    assert r_out.shape == x_out.shape == (0, 64)
    ids, wt = moe.moe_select_experts(e(0, 8, device="cuda"), 2)
    assert ids.shape == wt.shape == (0, 2)
    out = moe.moe_adapter_add(y, y, e(1, 8, 64, dtype=BF, device="cuda"), e(1, 64, 8, dtype=BF, device="cuda"), torch.ones(1, device="cuda"),
                              torch.zeros(1, dtype=torch.int32, device="cuda"), e(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 64)
