"""GPU: infinite values in a bf16 cache under moe_paged_attention, in every place of a request."""
import math

import pytest
import torch

from test_attention_ops import BF, Batch, attention_ref, gen, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens,n_q,window", [([1], [1], 2, 0), ([1, 1], [80, 300], 4, 0), ([3, 1], [500, 70], 6, 0), ([1, 2], [900, 40], 4, 333),
                                                 ([1], [20011], 2, 0), ([16], [700], 8, 0)])
def test_infinite_values_have_their_weight_everywhere(m, D, new, lens, n_q, window):  # noqa: F811
    """Infinities among the values of a bf16 cache, anywhere: one that a row sees makes its column infinite, two of both signs NaN;
    the other columns and rows are as if they were not there."""
    b = Batch(41 + D, new, lens, 2, D, 16).fill(std=0.5)
    rng = gen(D)
    marks = []  # request, token, head, column, value
    for s, l in enumerate(lens):
        for x in range(24):
            t, c = (int(torch.randint(n, (1,), generator=rng, device="cuda")) for n in (l, D))
            marks.append((s, t, x % 2, c, math.inf if x % 3 else -math.inf))
        marks += [(s, l - 1, 0, 1, math.inf), (s, l - 1, 1, D - 1, -math.inf)]
    q = b.normal(b.T, n_q, D, std=1.5).to(BF)
    ref, _, tol, _ = attention_ref(b, q, D ** -0.5, window)
    for s, t, h, c, value in marks:
        x = b.got(b.v_cache, s, [t])
        x[0, h, c] = value
        b.put(b.v_cache, s, [t], x)
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=max(new), window=window)
    m.moe_read_device_status()
    group, want = n_q // 2, ref.clone()
    held = {}
    for s, t, h, c, value in marks:
        held[s, t, h, c] = value
    for (s, t, h, c), value in held.items():
        for i in range(new[s]):
            pos = lens[s] - new[s] + i
            if t <= pos and (not window or t > pos - window):
                want[b.off[s] + i, h * group:(h + 1) * group, c] += value
    assert bool(want.isinf().any()) and bool(want.isfinite().any())
    odd = ~want.isfinite()
    assert torch.equal(torch.nan_to_num(out.double(), 7.0, 8.0, 9.0)[odd], torch.nan_to_num(want, 7.0, 8.0, 9.0)[odd])
    assert bool(((out.double() - want).abs() <= tol)[~odd].all())
