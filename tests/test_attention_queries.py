"""GPU: moe_paged_attention's queries near the largest numbers of their type."""
import pytest
import torch

from test_attention_ops import BF, E4M3, Batch, attention_ref, gen, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,top", [(BF, 2.0 ** 120), (BF, 2.0 ** 123)] + [(E4M3, 2.0 ** e) for e in (120, 123, 124, 125, 126, 127)])
def test_queries_near_the_top_of_their_type(m, dtype, top):  # noqa: F811
    # (of a bf16 cache q . k is an FP32 sum as it is, below 64 x 0.25 x 2^124 = 2^128 at the two sizes; of an 8-bit cache it is a
    # sum of q's codes, and any finite q is a number)
    b = Batch(42, [1, 2], [300, 70], 1, 64, 16, dtype).fill(std=0.1)
    b.k_scale = b.v_scale = None  # (keys and values are the codes)
    q = ((torch.rand(3, 4, 64, generator=gen(3), device="cuda") + 1.0) * top * (1 - 2.0 ** -9)).to(BF)
    q = torch.where(torch.rand(3, 4, 64, generator=gen(4), device="cuda") < 0.5, q, -q)
    for s, l in enumerate(b.lens):
        b.put(b.k_cache, s, range(l), (b.normal(l, 1, 64) * 0.0625).to(dtype))
    scale = 1.0 / top
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, scale=scale)
    m.moe_read_device_status()
    ref, _, tol, _ = attention_ref(b, q, scale, 0)
    assert bool(out.isfinite().all()) and bool(((out.double() - ref).abs() <= tol).all())
