"""GPU: the softmax weights of moe_paged_attention where they are small beside the largest, against the formula in 64 bits."""
import math

import pytest
import torch

from test_attention_ops import BF, E4M3, U32, Batch, ints, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("S,L,new", [(400, 2000, 1), (3, 60, 1), (40, 3000, 2), (1, 40003, 1)])
@pytest.mark.parametrize("below", [12, 20, 24, 26, 32])
def test_many_small_weights_beside_a_large_one(m, dtype, S, L, new, below):  # noqa: F811
    """The first token outweighs each of the others by 2^below and has the value 0: the others are the output."""
    D, page = 64, 16
    b = Batch(40, [new], [L], 1, D, page, dtype).fill()
    one = torch.zeros(L, 1, D, device="cuda")
    one[0, 0, 0] = 1.0
    b.put(b.k_cache, 0, range(L), one.to(dtype))
    v = b.normal(L, 1, D) * 0.1 + 1.0
    v[0] = 0.0
    b.put(b.v_cache, 0, range(L), (v if dtype is BF else v / b.v_scale[:, None]).to(dtype))
    # every request reads the same pages; the first token's score is below * ln 2, the others' are 0
    q = torch.zeros(S * new, 2, D, device="cuda")
    q[:, 0, 0], q[:, 1, 0] = below, below - 0.5
    q = q.to(BF)
    scale = math.log(2) / (1.0 if b.k_scale is None else float(b.k_scale))
    lse = torch.empty(S * new, 2, device="cuda")
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, ints(list(range(0, S * new + 1, new))), ints([L] * S), b.pages.expand(S, -1).contiguous(),
                                max_new=new, scale=scale, k_scale=b.k_scale, v_scale=b.v_scale, lse=lse)
    m.moe_read_device_status()
    vv = b.values(0)[1][:, 0]
    for i in range(new):
        n = L - new + i + 1
        for j in range(2):
            d = float(q[i, j, 0])
            z = torch.zeros(n, dtype=torch.float64, device="cuda")
            z[0] = math.log(2) * d
            p = torch.softmax(z, 0)
            want, size = p @ vv[:n], p @ vv[:n].abs()
            # the largest score is off by its few FP32 roundings, a weight by twice that and the exponential's 2^-22; the
            # weights by their rounding: 2^-16 (two bf16 values) or 2^-11 (FP16), the FP16 ones, held as parts of 2^-15 of the
            # largest, by 2^-25 of that at the least (2^-40); sums of n terms; the output's rounding
            delta = 2 * (8 * U32 * math.log(2) * d + 2.0 ** -22)
            rel = 2 * delta + (2.0 ** -16 if dtype is BF else 2.0 ** -11) + 2 * (n + 16) * U32
            tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (size * rel + (0 if dtype is BF else n * 2.0 ** -40 * float(p.max()) * vv.abs().max()))
            got = out[i::new, j].double()
            assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / want.abs()).max())
            assert bool(((lse[i::new, j].double() - torch.logsumexp(z, 0)).abs() <= delta + 2 * (n + 16) * U32 + 8 * U32 * d).all())


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_keep_their_bits_where_values_cancel(m, dtype, D):  # noqa: F811
    """Few tokens of weights of one size and values of both signs: the bf16 output shows the weights' own bits where the sum is
    small beside its terms."""
    S, L, page = 400, 16, 16
    b = Batch(43, [1], [L], 1, D, page, dtype).fill()
    v = torch.where(b.normal(L, 1, D) > 0, 1.0, -1.0) * (1 + torch.randint(8, (L, 1, D), generator=b.g, device="cuda") / 8)
    b.put(b.v_cache, 0, range(L), (v * 16).to(dtype))
    if dtype is E4M3:
        b.v_scale.fill_(1.0 / 16)
    q = b.normal(S, 4, D, std=0.1).to(BF)
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, ints(list(range(S + 1))), ints([L] * S), b.pages.expand(S, -1).contiguous(),
                                k_scale=b.k_scale, v_scale=b.v_scale)
    m.moe_read_device_status()
    kk, vv = (x[:, 0] for x in b.values(0))
    z = q.double() @ kk.T * D ** -0.5
    p = torch.softmax(z, 2)
    want, size = p @ vv, p @ vv.abs()
    top = float(((q.double().abs() @ kk.abs().T) * D ** -0.5).max())
    # scores off by their sums' roundings, weights by twice that, the exponential's 2^-22 and their own 2^-16 or 2^-22 (and
    # 2^-40), sums of 16, the output's rounding
    delta = 2 * ((D + 8) * U32 * top + 2.0 ** -22)
    tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * size * (2 * delta + (2.0 ** -16 if dtype is BF else 2.0 ** -21) + 2 * 32 * U32)
    assert bool((want.abs() < 2.0 ** -8 * size).any())
    assert bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() / size).max())
