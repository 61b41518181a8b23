"""Host-side check of moe_cache_append: keys and values that lie on one another are refused, exactly those (no GPU)."""
import random

import numpy as np
import pytest

from test_attention_refusals import INVALID, MB, append, cache, m, no_gpu  # noqa: F401

K = 100 * MB
# (dtype, pages, page, n_kv, D, strides in elements)
LAYOUTS = [
    (0, 8, 16, 2, 128, (16 * 2 * 128, 2 * 128, 128)),
    (0, 8, 16, 2, 128, (16 * 2 * 128, 128, 16 * 128)),            # heads first
    (2, 8, 16, 2, 64, (2 * 16 * 2 * 64, 2 * 64, 64)),             # pages twice as far apart
    (0, 5, 8, 3, 64, (3 * 64, 5 * 3 * 64, 64)),                   # pages innermost but heads
    (0, 1, 16, 1, 64, (0, 64, 0)),
    (2, 3, 4, 2, 64, (4 * 2 * 192 + 32, 2 * 192, 192)),           # gaps behind every head
]


def call(m, layout, apart):  # noqa: F811
    dtype, n_pages, page, n_kv, D, ld = layout
    return append(m, C=cache(m, dtype, n_pages, page, n_kv, D, k=K, v=K + apart, ld=ld), q=None, out=None, n_q=0, w_q=None, rot=16,
                  ld_k=n_kv * D, ld_v=n_kv * D, ws=None)


def places(layout):
    _, n_pages, page, n_kv, D, ld = layout
    i = np.indices((n_pages, page, n_kv, D))
    return i[0] * ld[0] + i[1] * ld[1] + i[2] * ld[2] + i[3]


@pytest.mark.parametrize("layout", LAYOUTS)
def test_places_that_meet(m, layout):  # noqa: F811
    es = 1 if layout[0] == 2 else 2
    at = places(layout).ravel()
    held = set(at.tolist())
    assert len(held) == at.size
    span, step = int(at.max()) + 1, 16 // es
    rng = random.Random(1)
    shifts = {0, span, -span} | {s * step for s in range(-40, 40)} | {rng.randrange(-span // step - 2, span // step + 2) * step for _ in range(60)}
    shifts |= {sign * n * ld for ld in layout[5] for n in range(1, 4) for sign in (1, -1)}
    shifts |= {sign * (n * ld + o) for ld in layout[5] for n in (1, 2) for sign in (1, -1) for o in (step, -step)}
    found = set()
    for d in sorted(shifts):
        if d % step:
            continue
        want = bool(np.isin(at + d, at).any())
        found.add(want)
        assert call(m, layout, d * es) == INVALID
        text = m.lib().moe_last_error_detail()
        assert (b"lie on one another" in text) == want and (want or b"workspace" in text), (d, text)
    assert found == {True, False}


def test_turns_of_keys_and_values_are_taken(m, no_gpu):  # noqa: F811
    from test_attention_refusals import NO_DEVICE

    def ok(layout, apart):
        dtype, n_pages, page, n_kv, D, ld = layout
        return append(m, C=cache(m, dtype, n_pages, page, n_kv, D, k=K, v=K + apart, ld=ld)) == NO_DEVICE

    assert ok((0, 8, 16, 2, 128, (2 * 16 * 256, 256, 128)), 16 * 256 * 2)  # [pages, 2, slots, heads, D]
    assert ok((0, 8, 16, 2, 128, (16 * 512, 512, 128)), 512)               # [pages, slots, 2, heads, D]
    assert ok((0, 8, 16, 2, 128, (16 * 512, 512, 256)), 256)               # [pages, slots, heads, 2, D]
    assert ok((0, 8, 16, 2, 128, (16 * 512, 512, 256)), -256)
