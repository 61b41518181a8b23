"""GPU: FP8 encoding and products, cache appends with norm and rotation, and attention over a paged cache, each against its
formula in 64 bits. Slots of the cache that hold no token are filled with NaN, tables' unused places with ids far outside.

Tolerances count roundings: bf16 2^-8 of a value, FP32 2^-24, FP16 2^-11, E4M3 2^-4 (half a step each)."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    import nvfp4_w4a4_mixture_gb300 as m

    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Requests of `new` tokens each, `lens` with them, in a cache of random pages."""

    def __init__(self, seed, new, lens, n_kv, D, page, dtype=BF, heads_first=False, tail=0, from_pos=None):
        g, rng = gen(seed), random.Random(seed)
        self.new, self.lens, self.n_kv, self.D, self.page, self.dtype = new, lens, n_kv, D, page, dtype
        first = [0] * len(new) if from_pos is None else from_pos
        counts = [max(0, -(-l // page)) for l in lens]
        n_pages = sum(c - f // page for c, f in zip(counts, first)) + 3
        order = list(range(n_pages))
        rng.shuffle(order)
        width = max([1] + counts) + 1
        table, at = [], 0
        for c, f in zip(counts, first):
            head = f // page
            table.append([2 ** 30] * head + order[at: at + c - head] + [-7 - rng.randrange(5)] * (width - c))
            at += c - head
        self.table = table
        self.pages, self.kv_len = ints(table), ints(lens)
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        self.off = off
        self.offsets, self.T = ints(off), off[-1] + tail
        shape = (n_pages, n_kv, page, D) if heads_first else (n_pages, page, n_kv, D)

        def cache():
            v = torch.full(shape, float("nan"), dtype=torch.float32, device="cuda").to(dtype)
            return v.transpose(1, 2) if heads_first else v

        self.k_cache, self.v_cache = cache(), cache()
        self.k_scale = self.v_scale = None
        if dtype is E4M3:
            self.k_scale, self.v_scale = (torch.rand(n_kv, generator=g, device="cuda") * 0.02 + 0.01 for _ in range(2))
        self.g = g

    def normal(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.g, device="cuda") * std

    def fill(self, std=1.0):
        """Tokens in every place that the requests hold."""
        for s, l in enumerate(self.lens):
            for cache, scale in ((self.k_cache, self.k_scale), (self.v_cache, self.v_scale)):
                x = self.normal(max(l, 0), self.n_kv, self.D, std=std)
                if scale is not None:
                    x = (x / scale[:, None]).clamp(-448, 448)
                self.put(cache, s, range(l), x.to(self.dtype))
        return self

    def places(self, s, positions):
        p = torch.tensor(list(positions), dtype=torch.long, device="cuda")
        t = torch.tensor(self.table[s], device="cuda")
        return t[p // self.page], p % self.page

    def put(self, cache, s, positions, x):
        if len(positions):
            page, slot = self.places(s, positions)
            if cache.dtype is E4M3:
                cache, x = cache.view(torch.uint8), x.view(torch.uint8)
            cache[page, slot] = x

    def got(self, cache, s, positions):
        page, slot = self.places(s, positions)
        if cache.dtype is E4M3:
            return cache.view(torch.uint8)[page, slot].view(E4M3)
        return cache[page, slot]

    def values(self, s):
        """Keys and values of request s in 64 bits, [len, n_kv, D]."""
        out = []
        for cache, scale in ((self.k_cache, self.k_scale), (self.v_cache, self.v_scale)):
            x = self.got(cache, s, range(self.lens[s])).double()
            out.append(x if scale is None else x * scale.double()[:, None])
        return out

    def tables(self):
        return self.offsets, self.kv_len, self.pages


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def attention_ref(b, q, scale, window):
    """(out, lse, bound of the error) in 64 bits."""
    T, n_q, D = q.shape
    group = n_q // b.n_kv
    out = torch.zeros(T, n_q, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, n_q), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for s, (n, l) in enumerate(zip(b.new, b.lens)):
        if not n or not l:
            continue
        k, v = b.values(s)
        for i in range(n):
            pos = l - n + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            t = b.off[s] + i
            for j in range(n_q):
                kk, vv, qq = k[lo: pos + 1, j // group], v[lo: pos + 1, j // group], q[t, j].double()
                z = kk @ qq * scale
                p = torch.softmax(z, 0)
                out[t, j] = p @ vv
                lse[t, j] = torch.logsumexp(z, 0)
                # a score is off by its D products' and sums' roundings and those of its exponent's argument (in
                # powers of two), a weight by twice that (its own and the largest's) and the exponential's 2^-22
                N = pos + 1 - lo
                size = float(((kk.abs() @ qq.abs()) * abs(scale)).max())
                delta = 2 * ((D + 8) * U32 * size + 2.0 ** -22)
                # the weights' own rounding for the product (two bf16 values, or one FP16 value, whose smallest are 2^-25
                # off), sums of N terms in some order, and the rounding of the output
                # (the largest weight before normalisation is 1, so the sum is 1 at least)
                weight = 2.0 ** -16 if b.dtype is BF else 2.0 ** -11
                size_v = p @ vv.abs()
                tol[t, j] = 2.0 ** -8 * out[t, j].abs() + size_v * (2 * delta + weight + 2 * (N + 16) * U32) + 2.0 ** -133
                if b.dtype is E4M3:
                    tol[t, j] += N * 2.0 ** -25 * vv.abs().max()
                tol_lse[t, j] = delta + 2 * (N + 16) * U32 + 4 * U32 * (abs(float(lse[t, j])) + size)
    return out, lse, tol, tol_lse


def check_attention(m, b, n_q, max_new=None, scale=None, window=0, q_std=1.5, q=None):
    if q is None:
        q = b.normal(b.T, n_q, b.D, std=q_std).to(BF)
    out = torch.full_like(q, 7.0)
    lse = torch.full((b.T, n_q), 7.0, device="cuda")
    got = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=max_new or max([1] + b.new), scale=scale,
                                window=window, k_scale=b.k_scale, v_scale=b.v_scale, out=out, lse=lse)
    assert got is out
    m.moe_read_device_status()
    ref, ref_lse, tol, tol_lse = attention_ref(b, q, b.D ** -0.5 if scale is None else scale, window)
    live = b.off[-1]
    assert bool((out[live:] == 7.0).all()) and bool((lse[live:] == 7.0).all())  # rows behind the last request
    over = (out[:live].double() - ref[:live]).abs() - tol[:live]
    assert bool((over <= 0).all()), float(over.max())
    empty = ref_lse[:live] == -math.inf
    assert torch.equal(lse[:live] == -math.inf, empty)
    over = ((lse[:live].double() - ref_lse[:live]).abs() - tol_lse[:live])[~empty]
    assert bool((over <= 0).all()), float(over.max())
    return out, lse


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,lens,n_q,n_kv,page", [
    ([1], [1], 1, 1, 16),
    ([1], [64], 2, 1, 8),
    ([1, 1, 1], [63, 65, 129], 8, 2, 16),
    ([2, 0, 1, 3], [2, 5, 1, 200], 10, 2, 4),
    ([4], [700], 16, 2, 64),
    ([5, 8, 1], [5, 77, 300], 21, 3, 1),
    ([16, 3], [130, 3], 8, 1, 32),
])
def test_attention(m, dtype, D, new, lens, n_q, n_kv, page):
    check_attention(m, Batch(D + len(new), new, lens, n_kv, D, page, dtype, heads_first=page > 8, tail=3).fill(), n_q)


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 1000, 2 ** 31 - 1])
def test_attention_window(m, dtype, window):
    check_attention(m, Batch(window % 97, [1, 4, 2], [300, 129, 2], 2, 64, 16, dtype).fill(), 6, window=window)


@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_attention_rows_that_see_nothing(m, dtype):
    # idle slots, and a request whose first tokens have no place in the cache
    b = Batch(5, [1, 3, 1, 4, 1], [0, 70, 0, 2, 9], 2, 128, 16, dtype, tail=2).fill()
    check_attention(m, b, 8)
    check_attention(m, Batch(6, [1], [0], 1, 64, 16, dtype), 4)
    check_attention(m, Batch(6, [0, 0], [0, 40], 1, 64, 16, dtype, tail=3).fill(), 4)


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("window", [0, 7])
def test_attention_masked_places_hold_anything(m, dtype, window):
    # the later tokens of a verify window (and those before a window) are infinities and NaN: rows that do not see them
    # are as if they were not there, the others get what the arithmetic gives
    n, l, D = 4, 150, 64
    b = Batch(8, [n], [l], 1, D, 16, dtype).fill()
    q = b.normal(n, 3, D).to(BF)
    bad = torch.full((1, 1, D), float("nan"), device="cuda").to(dtype)
    if dtype is BF:
        bad[0, 0, ::2] = float("inf")
    places = [l - 2] + ([l - n - window + 1] if window else [])  # seen by the last two rows; by the first row alone
    for cache in (b.k_cache, b.v_cache):
        for pos in places:
            b.put(cache, 0, [pos], bad)
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=n, window=window, k_scale=b.k_scale, v_scale=b.v_scale)
    ref, _, tol, _ = attention_ref(b, q, D ** -0.5, window)
    clean = [i for i in range(n) if not any((l - n + i) - (window or l) < pos <= l - n + i for pos in places)]
    assert clean and len(clean) < n
    for i in range(n):
        if i in clean:
            assert bool(((out[i].double() - ref[i]).abs() <= tol[i]).all())
        else:
            assert bool(out[i].isnan().all())


def test_attention_infinite_values_that_are_seen(m):
    # an infinity among the values alone is seen with its weight by the rows that see it
    b = Batch(9, [3], [80], 1, 128, 16).fill()
    x = b.got(b.v_cache, 0, [78])
    x[0, 0, 5], x[0, 0, 6] = float("inf"), -float("inf")
    b.put(b.v_cache, 0, [78], x)
    q = b.normal(3, 2, 128).to(BF)
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=3)
    assert bool((out[1:, :, 5] == float("inf")).all()) and bool((out[1:, :, 6] == -float("inf")).all())
    ref, _, tol, _ = attention_ref(b, q, 128 ** -0.5, 0)
    keep = [c for c in range(128) if c not in (5, 6)]
    assert bool(((out.double() - ref).abs() <= tol)[:, :, keep].all()) and bool(out[0].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("q_std", [0.0, 1e-30, 40.0, 3e4])
def test_attention_scores_of_any_size(m, dtype, q_std):
    check_attention(m, Batch(11, [1, 2], [500, 90], 2, 128, 16, dtype).fill(), 4, q_std=q_std, scale=1e-3 if q_std > 100 else None)


def test_attention_lowest_values(m):
    # keys at the type's lowest value: scores near -3e38 are numbers like others, not masks
    b = Batch(12, [2], [70], 1, 64, 16).fill()
    low = torch.finfo(BF).min
    x = torch.zeros(1, 1, 64, device="cuda").to(BF)
    x[0, 0, 0] = low
    for pos in range(0, 70):
        b.put(b.k_cache, 0, [pos], x)
    q = torch.zeros(2, 2, 64, device="cuda").to(BF)
    q[:, :, 0] = 1.0
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, scale=0.5)
    _, v = b.values(0)
    for i, n in ((0, 69), (1, 70)):  # equal scores: the mean
        want = v[:n, 0].mean(0)
        assert bool(((out[i, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * v[:n, 0].abs().mean(0)).all())


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("new", [1, 3])
def test_attention_long_and_split(m, dtype, new):
    # one request over every multiprocessor, and beside it short ones
    check_attention(m, Batch(13, [new], [40003], 1, 64, 128, dtype).fill(), 2)
    check_attention(m, Batch(14, [new, 1, new, 1], [30011, 3, 9000, 64], 2, 128, 64, dtype).fill(), 4)


def test_attention_many_requests(m):
    rng = random.Random(1)
    S = 300
    new = [rng.choice((0, 1, 1, 1, 2)) for _ in range(S)]
    check_attention(m, Batch(15, new, [rng.choice((1, 2, 30, 64, 90, 200)) + 2 for _ in range(S)], 1, 64, 16, tail=1).fill(), 2)


def test_attention_rows_past_a_tile(m):
    # 16 new tokens of 64 query heads a key head: 1024 rows of one key head
    check_attention(m, Batch(16, [16, 2], [100, 70], 1, 64, 16).fill(), 64)


def test_attention_in_place_and_strided(m):
    b = Batch(17, [2, 1], [90, 33], 2, 64, 16).fill()
    wide = b.normal(3, 3 * 4 * 64).to(BF)
    q = wide[:, 256:512].view(3, 4, 64)
    ref = m.moe_paged_attention(q.contiguous(), b.k_cache, b.v_cache, *b.tables(), max_new=2)
    keep = wide.clone()
    assert m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=q) is q
    assert torch.equal(q, ref)
    keep[:, 256:512] = wide[:, 256:512]
    assert torch.equal(wide, keep)


def test_attention_of_one_buffer_of_keys_and_values(m):
    # [pages, 2, slots, heads, D]: keys and values by turns
    b = Batch(18, [1, 2], [90, 33], 2, 64, 16).fill()
    both = torch.stack((b.k_cache, b.v_cache), 1)
    q = b.normal(3, 4, 64).to(BF)
    ref = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2)
    assert torch.equal(ref, m.moe_paged_attention(q, both[:, 0], both[:, 1], *b.tables(), max_new=2))


def test_attention_at_the_last_positions(m):
    # the longest request, its table's rows one and the same page; a window keeps the work small
    D, page, W, n = 64, 65536, 100, 3
    g = gen(30)
    k, v = (torch.randn(1, page, 1, D, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(n, 2, D, generator=g, device="cuda").to(BF)
    pages = torch.zeros(1, 32768, dtype=torch.int32, device="cuda")
    last = 2 ** 31 - 65
    out = m.moe_paged_attention(q, k, v, ints([0, n]), ints([last]), pages, max_new=n, window=W)
    m.moe_read_device_status()
    for i in range(n):
        p = torch.arange(last - n + i - W + 1, last - n + i + 1, device="cuda") % page
        z = torch.einsum("hd,td->ht", q[i].double(), k[0, p, 0].double()) * D ** -0.5
        ref = torch.softmax(z, 1) @ v[0, p, 0].double()
        assert bool(((out[i].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * 4).all())
    with pytest.raises(m.MoeError):
        m.moe_paged_attention(q, k, v, ints([0, n]), ints([last + 1]), pages, max_new=n, window=W)
        m.moe_read_device_status()


@pytest.mark.parametrize("dtype", [BF, E4M3])
def test_offsets_past_32_bits(m, dtype):
    # pages 2^28 elements apart in one buffer: the last begins behind 2^32 elements
    D, page, n_pages = 64, 16, 18
    buf = torch.zeros(n_pages << 28, dtype=torch.uint8 if dtype is E4M3 else torch.int16, device="cuda").view(dtype)
    shape, strides = (n_pages, page, 1, D), (1 << 28, D, D, 1)
    b = Batch(31, [2, 1], [40, 33], 1, D, page, dtype)
    b.k_cache, b.v_cache = torch.as_strided(buf, shape, strides), torch.as_strided(buf, shape, strides, 1 << 20)
    b.table = [[17, 3, 16, 0], [5, 17 - 2, 14, 0]]
    b.pages = ints(b.table)
    b.fill()
    q, k, v = (b.normal(3, h, D).to(BF) for h in (4, 1, 1))
    m.moe_cache_append(None, k, v, b.k_cache, b.v_cache, *b.tables(), k_scale=b.k_scale, v_scale=b.v_scale)
    for s, rows in ((0, slice(0, 2)), (1, slice(2, 3))):
        places = range(b.lens[s] - b.new[s], b.lens[s])
        want = v[rows] if dtype is BF else (v[rows].float() / b.v_scale[:, None]).clamp(-448, 448).to(E4M3)
        assert torch.equal(b.got(b.v_cache, s, places).float(), want.float())
    check_attention(m, b, 4, q=q)


def test_attention_repeats_itself_and_in_a_graph(m):
    b = Batch(19, [1, 2, 1], [5000, 333, 64], 2, 128, 16).fill()
    q = b.normal(4, 8, 128).to(BF)
    call = lambda out: m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=out)  # noqa: E731
    first, second = call(torch.empty_like(q)), call(torch.empty_like(q))
    assert torch.equal(first, second)
    outs = [torch.empty_like(q) for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):  # two graphs at the same time, each with its own workspace
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    # the tables are read at replay
    b.kv_len.copy_(ints([4000, 300, 0]))
    b.lens = [4000, 300, 0]
    graphs[0].replay()
    torch.cuda.synchronize()
    ref, _, tol, _ = attention_ref(b, q, 128 ** -0.5, 0)
    assert bool(((outs[0].double() - ref).abs() <= tol).all())


def test_attention_two_streams(m):
    b = Batch(20, [1] * 5, [3000, 10, 700, 64, 1], 2, 64, 16).fill()
    q = b.normal(5, 8, 64).to(BF)
    ref = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables())
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables()))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_attention_broken_tables_are_reported(m):
    b = Batch(21, [1, 1, 2], [40, 50, 60], 1, 64, 16, tail=1).fill()
    q = b.normal(5, 2, 64).to(BF)
    good = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=2, out=torch.full_like(q, 7.0))
    ws = m.Workspace(m.moe_attention_workspace_bytes(3, 2, 1, 64, 2))

    def call(offsets=b.offsets, kv_len=b.kv_len, pages=b.pages, max_new=2):
        out = m.moe_paged_attention(q, b.k_cache, b.v_cache, offsets, kv_len, pages, max_new=max_new, out=torch.full_like(q, 7.0), ws=ws)
        with pytest.raises(m.MoeError):
            m.moe_read_device_status(ws)
        return out

    seven = torch.full_like(q[0], 7.0)
    out = call(kv_len=ints([40, -1, 60]))
    assert torch.equal(out[0], good[0]) and torch.equal(out[1], seven) and torch.equal(out[2:], good[2:])
    out = call(kv_len=ints([40, 10 ** 6, 60]))
    assert torch.equal(out[1], seven) and torch.equal(out[2:], good[2:])
    out = call(max_new=1)
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[2], seven) and torch.equal(out[3], seven)
    call(offsets=ints([0, 3, 2, 4]))
    call(offsets=ints([0, 1, 2, 9]))
    call(offsets=ints([1, 1, 2, 4]))
    for page in (-1, 10 ** 9, b.k_cache.shape[0]):
        t = b.pages.clone()
        t[1, 0] = page
        out = call(pages=t)
        assert torch.equal(out[0], good[0]) and torch.equal(out[2:], good[2:])
    m.moe_read_device_status(ws)


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_out_of_order_take_no_row_behind_their_begin(m, D):
    """Offsets in which a search for row 4's request ends at one that begins behind it."""
    b = Batch(57, [5, 1, 1, 0, 1], [300, 290, 280, 16, 270], 1, D, 16).fill()
    wrong = ints([0, 5, 6, 7, 1, 2])
    q = b.normal(8, 4, D).to(BF)
    good = m.moe_paged_attention(q, b.k_cache, b.v_cache, *b.tables(), max_new=5)
    ws = m.Workspace(m.moe_attention_workspace_bytes(5, 4, 1, D, 5))
    out = m.moe_paged_attention(q, b.k_cache, b.v_cache, wrong, b.kv_len, b.pages, max_new=5, out=torch.full_like(q, 7.0), ws=ws)
    with pytest.raises(m.MoeError):
        m.moe_read_device_status(ws)
    seven = torch.full_like(q[0], 7.0)
    for t in (0, 2, 3, 4, 5, 6):  # (row 1 is two requests')
        assert torch.equal(out[t], good[t]) or torch.equal(out[t], seven), t
    assert torch.equal(out[7], seven)

    k, v = (b.normal(8, 1, D).to(BF) for _ in range(2))
    before = [[b.got(c, s, range(b.lens[s] - n)) for c in (b.k_cache, b.v_cache)] for s, n in enumerate(b.new)]
    m.moe_cache_append(None, k, v, b.k_cache, b.v_cache, wrong, b.kv_len, b.pages, ws=ws)
    with pytest.raises(m.MoeError):
        m.moe_read_device_status(ws)
    for s, n in enumerate(b.new):  # what lies before a request's new tokens stays
        for c, was in zip((b.k_cache, b.v_cache), before[s]):
            assert torch.equal(b.got(c, s, range(b.lens[s] - n)), was), s


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
def append_ref(b, q, k, inv, interleaved, w_q, w_k, eps, off):
    """Queries and keys in 64 bits with the size of the terms that each is a sum of."""
    T = b.off[-1]
    pos = torch.tensor([l - n + i for n, l in zip(b.new, b.lens) for i in range(n)], dtype=torch.float64, device="cuda")
    out = []
    for x, w in ((q, w_q), (k, w_k)):
        x = x[:T].double()
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (w.double() + off)
        x = x.clone()
        size = x.abs()
        if inv is not None:
            h = inv.numel()
            a, c = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
            ang = (pos[:, None] * inv.double())[:, None]
            xa, xc = x[..., a].clone(), x[..., c].clone()
            x[..., a], x[..., c] = xa * ang.cos() - xc * ang.sin(), xa * ang.sin() + xc * ang.cos()
            size[..., a] = size[..., c] = xa.abs() + xc.abs()
        out.append((x, size))
    return out


@pytest.mark.parametrize("dtype", [BF, E4M3])
@pytest.mark.parametrize("D,rot,interleaved,norm,n_q,n_kv,page,new,lens", [
    (64, 64, False, True, 4, 2, 16, [1], [1]),
    (64, 16, True, False, 1, 1, 8, [3, 1], [5, 100001]),
    (128, 128, False, True, 7, 1, 1, [1, 0, 5, 2], [70000, 9, 5, 64]),
    (128, 96, True, True, 32, 4, 32, [40, 1, 1], [41, 17, 1]),
    (256, 64, False, True, 16, 2, 64, [4], [2 ** 20 + 3]),
    (256, 256, False, False, 3, 3, 4, [130, 2], [130, 2 ** 18]),
    (256, 0, False, True, 2, 2, 16, [9], [20]),
    (64, 48, False, False, 0, 5, 16, [3], [3]),
])
def test_append(m, dtype, D, rot, interleaved, norm, n_q, n_kv, page, new, lens):
    b = Batch(D + rot, new, lens, n_kv, D, page, dtype, heads_first=n_kv > 2, tail=2,
              from_pos=[l - n for n, l in zip(new, lens)])
    qkv = b.normal(b.T, (n_q + 2 * n_kv) * D, std=2.0).to(BF)
    q, k, v = (x.view(b.T, -1, D) for x in qkv.split((n_q * D, n_kv * D, n_kv * D), 1))
    inv = None if rot == 0 else (1e6 if D == 256 else 1e4) ** (-torch.arange(0, rot, 2, device="cuda").float() / rot)
    w_q, w_k = ((1 + b.normal(D, std=0.1)).to(BF) if norm else None for _ in range(2))
    before = b.k_cache.clone(), b.v_cache.clone()
    out = torch.full((b.T, n_q, D), 7.0, device="cuda").to(BF) if n_q else None
    got = m.moe_cache_append(q if n_q else None, k, v, b.k_cache, b.v_cache, *b.tables(), inv_freq=inv, interleaved=interleaved,
                             w_q=w_q if n_q else None, w_k=w_k, eps=1e-5, w_offset=0.25, k_scale=b.k_scale, v_scale=b.v_scale, out=out)
    m.moe_read_device_status()
    assert got is out
    live = b.off[-1]
    (rq, sq), (rk, sk) = append_ref(b, q if n_q else k, k, inv, interleaved, w_q, w_k, 1e-5, 0.25)
    # in FP32: the norm's sum of D squares (half of its relative error in the root), its root, products and weight, the
    # cosine and sine (2 units), their angle (2^-30 turns, and a unit of FP32 of half a turn), products and their sum
    near = ((D / 2 + 6) * norm + 8) * U32 + 2 * math.pi * 2.0 ** -30 + math.pi * U32
    if n_q:
        assert bool((out[live:] == 7.0).all())
        assert bool(((out[:live].double() - rq).abs() <= 2.0 ** -8 * rq.abs() + near * (1 + 2.0 ** -8) * sq).all())
    for s, (n, l) in enumerate(zip(new, lens)):
        if not n:
            continue
        rows, places = slice(b.off[s], b.off[s] + n), range(l - n, l)
        kk, vv = b.got(b.k_cache, s, places).double(), b.got(b.v_cache, s, places)
        if dtype is BF:
            assert bool(((kk - rk[rows]).abs() <= 2.0 ** -8 * rk[rows].abs() + near * (1 + 2.0 ** -8) * sk[rows]).all())
            assert torch.equal(vv, v[rows])
        else:
            ks = b.k_scale.double()[:, None]
            want, size = rk[rows] / ks, sk[rows] / ks
            # half a step of E4M3 (2^-10 the least); the rest moves a value by its own size before it is rounded
            assert bool(((kk - want.clamp(-448, 448)).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + (near + 2 * U32) * (1 + 2.0 ** -4) * size).all())
            assert torch.equal(vv.float(), (v[rows].float() / b.v_scale[:, None]).clamp(-448, 448).to(E4M3).float())
        for cache in (b.k_cache, b.v_cache):  # taken out for the comparison of all the rest
            b.put(cache, s, places, torch.zeros(n, n_kv, D, device="cuda").to(dtype))
        for cache in before:
            b.put(cache, s, places, torch.zeros(n, n_kv, D, device="cuda").to(dtype))
    view = torch.int16 if dtype is BF else torch.uint8
    assert torch.equal(b.k_cache.view(view), before[0].view(view)) and torch.equal(b.v_cache.view(view), before[1].view(view))


def test_append_far_positions_turn_exactly(m):
    # inv_freq 1: the angle is the position itself, modulo a turn, up to the longest of them
    D, places = 64, [2 ** 31 - 2, 2 ** 30 + 1, 10 ** 9, 12345677, 1]
    b = Batch(3, [1] * 5, [7] * 5, 1, D, 8)
    b.kv_len = ints([p + 1 for p in places])
    # every position in page 0: a table that wide would not fit, so its rows are the same memory
    page = 65536
    cache = torch.zeros(1, page, 1, D, device="cuda").to(BF)
    table = torch.zeros(1, 32768, dtype=torch.int32, device="cuda").expand(5, 32768).contiguous()
    q = torch.zeros(5, 1, D, device="cuda").to(BF)
    q[:, :, 0] = 1.0
    inv = torch.ones(D // 2, device="cuda")
    out = m.moe_cache_append(q, q.clone(), q.clone(), cache, cache.clone(), b.offsets, b.kv_len, table, inv_freq=inv)
    m.moe_read_device_status()
    p = torch.tensor(places, dtype=torch.float64, device="cuda")
    # inv_freq / 2 pi is held to 2^-54 of a turn: at position 2^31 that is 2^-23 of one
    tol = 2 * math.pi * (p * 2.0 ** -54 + 2.0 ** -30) + 2.0 ** -22
    for c, want in ((0, p.cos()), (D // 2, p.sin())):
        assert bool(((out[:, 0, c].double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all())


def test_append_in_place_and_special_values(m):
    b = Batch(22, [2, 1], [10, 33], 2, 64, 16)
    q, k, v = (b.normal(3, 2, 64).to(BF) for _ in range(3))
    v[0, 0, 3], v[1, 1, 5], k[2, 0, 63], q[0, 1, 40] = float("inf"), float("nan"), float("-inf"), float("nan")
    inv = 1e4 ** (-torch.arange(0, 32, 2, device="cuda").float() / 32)
    ref = m.moe_cache_append(q, k, v, b.k_cache, b.v_cache, *b.tables(), inv_freq=inv)
    caches = b.k_cache.clone(), b.v_cache.clone()
    assert m.moe_cache_append(q, k, v, b.k_cache, b.v_cache, *b.tables(), inv_freq=inv, out=q) is q
    assert torch.equal(q.view(torch.int16), ref.view(torch.int16))
    assert all(torch.equal(a.view(torch.int16), c.view(torch.int16)) for a, c in zip(caches, (b.k_cache, b.v_cache)))
    assert bool(q[0, 1, 40].isnan()) and bool(q[0, 1, :40].isfinite().all())
    assert torch.equal(b.got(b.v_cache, 0, [8, 9]).view(torch.int16), v[:2].view(torch.int16))
    # 8 bits: an infinity is the largest value, NaN stays
    e = Batch(22, [2, 1], [10, 33], 2, 64, 16, E4M3)
    m.moe_cache_append(None, k, v, e.k_cache, e.v_cache, *e.tables())
    got = e.got(e.v_cache, 0, [8, 9]).float()
    assert float(got[0, 0, 3]) == 448.0 and bool(got[1, 1, 5].isnan()) and float(e.got(e.k_cache, 1, [32]).float()[0, 0, 63]) == -448.0


def test_append_skips_what_has_no_place(m):
    b = Batch(23, [1, 3, 2], [0, 2, 40], 1, 64, 16, tail=1)
    q, k, v = (b.normal(7, 1, 64).to(BF) for _ in range(3))
    out = torch.full_like(q, 7.0)
    m.moe_cache_append(q, k, v, b.k_cache, b.v_cache, *b.tables(), out=out)
    m.moe_read_device_status()
    seven = torch.full_like(q[0], 7.0)
    assert torch.equal(out[0], seven) and torch.equal(out[1], seven) and torch.equal(out[6], seven)
    assert torch.equal(out[2:6], q[2:6])
    assert torch.equal(b.got(b.k_cache, 1, [0, 1]), k[2:4]) and torch.equal(b.got(b.v_cache, 2, [38, 39]), v[4:6])
    assert int(b.k_cache.isfinite().any(-1).sum()) == 4


def test_append_broken_tables_are_reported(m):
    b = Batch(24, [1, 2, 1], [40, 50, 60], 1, 64, 16)
    q, k, v = (b.normal(4, 1, 64).to(BF) for _ in range(3))
    ws = m.Workspace(4096)

    def call(offsets=b.offsets, kv_len=b.kv_len, pages=b.pages):
        out = m.moe_cache_append(q, k, v, b.k_cache, b.v_cache, offsets, kv_len, pages, out=torch.full_like(q, 7.0), ws=ws)
        with pytest.raises(m.MoeError):
            m.moe_read_device_status(ws)
        return out

    def rows(out):
        return [bool((out[t] != 7.0).any()) for t in range(4)]

    assert rows(call(kv_len=ints([40, 10 ** 6, 60]))) == [True, False, False, True]
    assert rows(call(kv_len=ints([40, -5, 60]))) == [True, False, False, True]
    call(offsets=ints([0, 3, 1, 4]))
    call(offsets=ints([0, 1, 3, 5]))
    call(offsets=ints([-1, 1, 3, 4]))
    # (a request that keeps the rules is appended beside one that breaks them: nothing outside the tables' pages)
    listed = sorted({p for row in b.table for p in row if p >= 0})
    other = [p for p in range(b.k_cache.shape[0]) if p not in listed]
    assert other and not bool(b.k_cache[other].isfinite().any()) and not bool(b.v_cache[other].isfinite().any())
    t = b.pages.clone()
    for page in (-1, 10 ** 9, b.k_cache.shape[0]):
        t[1, 3] = page
        call(pages=t)
    m.moe_read_device_status(ws)


def test_append_then_attention(m):
    """A decode step and a verify window after a prompt: the cache filled call by call gives what the whole sequence gives."""
    D, n_q, n_kv, page, rot = 128, 8, 2, 16, 64
    inv = 1e4 ** (-torch.arange(0, rot, 2, device="cuda").float() / rot)
    lens = [70, 33]
    b = Batch(25, [0, 0], lens, n_kv, D, page)
    xs = [[b.normal(l, h, D).to(BF) for h in (n_q, n_kv, n_kv)] for l in lens]
    w = (1 + b.normal(D, std=0.1)).to(BF)
    done = [0, 0]
    outs = [[], []]
    for step in ([40, 20], [1, 1], [4, 0], [16, 1], [9, 11]):
        off = ints([0, step[0], step[0] + step[1]])
        ends = [d + n for d, n in zip(done, step)]
        q, k, v = (torch.cat([x[i][d:e] for x, d, e in zip(xs, done, ends)]) for i in range(3))
        q = m.moe_cache_append(q, k, v, b.k_cache, b.v_cache, off, ints(ends), b.pages, inv_freq=inv, w_q=w, w_k=w)
        if max(step) <= 16:
            o = m.moe_paged_attention(q, b.k_cache, b.v_cache, off, ints(ends), b.pages, max_new=16).split(step)
            for i in range(2):
                outs[i].append(o[i])
        done = ends
    m.moe_read_device_status()
    assert done == lens
    b.new, b.off = [30, 13], [0, 30, 43]
    q = torch.cat([x[0][l - n:] for x, l, n in zip(xs, lens, b.new)])
    (rq, _), _ = append_ref(b, q, q, inv, False, w, w, 1e-6, 0.0)
    ref, _, tol, _ = attention_ref(b, rq.to(BF), D ** -0.5, 0)  # (over the keys that the cache holds)
    got = torch.cat([torch.cat(o) for o in outs])
    # a query's element that rounds the other way: one bf16 step of it in the scores, |dz| <= 2^-7 |q| |k| scale at most
    # for all; a few do, by chance, so the bar is that of the whole vector: 2^-7 of the weights' spread
    assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -7
    assert bool(((got.double() - ref).abs() <= tol + 2.0 ** -7 * 4).all())


# ------------------------------------------------------------------------------------------------
# FP8
# ------------------------------------------------------------------------------------------------
def quant_ref(x):
    T, K = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(T, -1, 128)
    most = p.abs().amax(2)
    scale = torch.where(most == 0, torch.ones_like(most), most / torch.full_like(most, 448.0))
    return (p / scale[:, :, None]).clamp(-448, 448).view(T, -1)[:, :K].to(E4M3), scale


@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (5, 2048), (130, 2064), (1000, 272), (7, 65536)])
def test_quantize_fp8_is_exact(m, T, K):
    x = (torch.randn(T, K, generator=gen(T + K), device="cuda") * torch.exp(torch.randn(T, 1, generator=gen(K), device="cuda") * 4)).to(BF)
    x[0, :16] = 0.0
    if T > 2:
        x[1] = 0.0
        x[2, 0], x[2, 5] = torch.finfo(BF).max, torch.finfo(BF).tiny
    wide = torch.zeros(T, K + 24, device="cuda").to(BF)
    wide[:, 8: K + 8] = x
    codes, scale = m.moe_quantize_fp8(wide[:, 8: K + 8])
    ref, ref_scale = quant_ref(x)
    assert torch.equal(scale, ref_scale) and torch.equal(codes.view(torch.uint8), ref.view(torch.uint8))


def test_quantize_fp8_special_values(m):
    x = torch.randn(3, 256, generator=gen(1), device="cuda").to(BF)
    x[0, 7], x[1, 200] = float("nan"), float("inf")
    codes, scale = m.moe_quantize_fp8(x)
    c = codes.float()
    assert bool(scale[0, 0].isnan()) and bool(c[0, :128].isnan().all()) and bool(c[0, 128:].isfinite().all())
    assert float(scale[1, 1]) == float("inf") and bool(c[1, 200].isnan()) and bool((c[1, 128:200] == 0).all())
    assert bool(scale[2].isfinite().all()) and bool(c[2].isfinite().all())


def gemm_case(T, N, K, seed):
    g = gen(seed)
    a = (torch.randn(T, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
    b = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(E4M3)
    sa = torch.exp(torch.randn(T, -(-K // 128), generator=g, device="cuda"))
    sb = torch.exp(torch.randn(-(-N // 128), -(-K // 128), generator=g, device="cuda"))
    return a, sa, b, sb


def gemm_ref(a, sa, b, sb):
    K, N = a.shape[1], b.shape[0]
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    w = b.double() * sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ w.T, x.abs() @ w.abs().T


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,N,K", [
    (1, 8, 16), (1, 128, 128), (4, 256, 2048), (3, 136, 272), (15, 1000, 144), (17, 512, 1040), (32, 264, 4096), (33, 128, 256),
    (64, 2048, 384), (65, 392, 640), (130, 1032, 272), (300, 640, 2048), (1000, 2056, 528), (2100, 2048, 256), (129, 20000, 144),
    (1, 40000, 160), (5, 128, 65536)])
def test_gemm_fp8(m, T, N, K, f32):
    a, sa, b, sb = gemm_case(T, N, K, T + N + K)
    wide = torch.full((T + 1, N + 16), 7.0, device="cuda").to(torch.float32 if f32 else BF)
    out = wide[:T, 8: N + 8]
    assert m.moe_gemm_fp8(a, sa, b, sb, out=out) is out
    m.moe_read_device_status()
    ref, size = gemm_ref(a, sa, b, sb)
    # products of codes are exact; a block's 128 are summed in FP32 (by the tensor core, which cuts instead of rounding:
    # a whole unit each), the blocks' sums are scaled (the product of the scales, and with it) and added
    tol = (2 * 128 + 2 * -(-K // 128) + 4) * U32 * size
    if not f32:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    over = (out.double() - ref).abs() - tol
    assert bool((over <= 0).all()), float(over.max())
    out.fill_(7.0)
    assert bool((wide == 7.0).all())  # nothing beside it


def test_gemm_fp8_of_quantized_rows(m):
    # a projection as a block makes it: encode, multiply
    x = torch.randn(70, 2048, generator=gen(5), device="cuda").to(BF)
    w = torch.randn(640, 2048, generator=gen(6), device="cuda") * 0.02
    sb = w.view(5, 128, 16, 128).abs().amax((1, 3)) / 448
    b = (w.view(5, 128, 16, 128) / sb[:, None, :, None]).view(640, 2048).to(E4M3)
    codes, sa = m.moe_quantize_fp8(x)
    out = m.moe_gemm_fp8(codes, sa, b, sb)
    m.moe_read_device_status()
    ref = x.double() @ w.double().T
    # two roundings to E4M3 of 2^-4 at most: errors of independent signs, their size 2^-4 / sqrt(3) each at the most
    assert float((out.double() - ref).norm() / ref.norm()) <= 2.0 ** -4


def test_gemm_fp8_special_values_stay_in_their_rows(m):
    for T in (4, 40, 2100):
        a, sa, b, sb = gemm_case(T, 2048, 256, T)
        want = m.moe_gemm_fp8(a, sa, b, sb)
        a[1, 3] = float("nan")
        sa[2, 1] = float("inf")
        got = m.moe_gemm_fp8(a, sa, b, sb)
        keep = [t for t in range(T) if t not in (1, 2)]
        assert torch.equal(got[keep], want[keep]) and bool(got[1].isnan().all()) and not bool(got[2].isfinite().any())


def test_gemm_fp8_repeats_itself_and_in_a_graph(m):
    for T, N, K in ((4, 1024, 2048), (2100, 2048, 512)):
        a, sa, b, sb = gemm_case(T, N, K, 3)
        first = m.moe_gemm_fp8(a, sa, b, sb)
        out = torch.empty_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_gemm_fp8(a, sa, b, sb, out=out)
        for _ in range(3):
            out.zero_()
            g.replay()
            assert torch.equal(out, first)
