"""Cases of the attention half around the mixture-of-experts layer, as a server runs it: FP8 encoding of activations and
the projections' matrix product with a scale for each block of 128, norm, position rotation and appending of keys and
values to a paged cache, and attention of a few new tokens a request over that cache.

run() computes a case in plain torch operations, or with `own` through nvfp4_w4a4_mixture_gb300.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _append(T, S, n_q, n_kv, D, rot, page, past=0, cache="bf16", norm=False, interleaved=False, heads_first=False, **kw):
    return dict(op="append", T=T, S=S, n_q=n_q, n_kv=n_kv, D=D, rot=rot, page=page, past=past, cache=cache, norm=norm,
                interleaved=interleaved, heads_first=heads_first, **kw)


def _attend(S, L, n_q, n_kv, D, page, new=1, idle=0, window=0, cache="bf16", heads_first=False, **kw):
    return dict(op="attend", S=S, L=L, n_q=n_q, n_kv=n_kv, D=D, page=page, new=new, idle=idle, window=window, cache=cache,
                heads_first=heads_first, **kw)


def _quant(T, K, **kw):
    return dict(op="quant", T=T, K=K, **kw)


def _gemm(T, N, K, **kw):
    return dict(op="gemm", T=T, N=N, K=K, **kw)


def listed():
    return [
        # a decode step: the verify window of four tokens late in a long conversation, a quarter of each head rotated
        _append(4, 1, 16, 2, 256, 64, 64, past=130000, norm=True, name="append 4 tokens"),
        # a full decode batch on an 8-bit cache, one token a request, pages with the heads first
        _append(256, 256, 32, 4, 128, 128, 16, past=20000, cache="e4m3", norm=True, heads_first=True,
                name="append 256 requests e4m3"),
        # ragged prompts and decode steps mixed, small heads, pairs of neighbours rotated, no norm
        _append(12365, 37, 14, 2, 64, 64, 32, past=900, interleaved=True, name="append 12365 mixed"),
        # a long prefill chunk
        _append(16384, 2, 16, 2, 256, 64, 64, past=16384, norm=True, name="append 16384 tokens"),
        # a decode step: the verify window of four tokens over one conversation
        _attend(1, 4100, 16, 2, 256, 64, new=4, name="attend 4 tokens over 4100"),
        # a full decode batch of ragged lengths
        _attend(64, 8192, 32, 8, 128, 16, name="attend 64 requests to 8192"),
        # one request with a whole code base in an 8-bit cache
        _attend(1, 300001, 16, 2, 256, 64, cache="e4m3", name="attend 1 over 300001 e4m3"),
        # a sliding-window layer: verify windows of one to three tokens, seven heads a key head, idle slots in the batch
        _attend(200, 6000, 14, 2, 64, 32, new=3, idle=9, window=1024, heads_first=True, name="attend 200 windows of 1024"),
        # a decode step's activations
        _quant(4, 2048, name="quant 4x2048"),
        # a long prefill chunk, the last block of a row short
        _quant(16384, 2064, name="quant 16384x2064"),
        # a decode step's projection to queries, keys and values
        _gemm(4, 5120, 2048, name="gemm 4x5120x2048"),
        # a long prefill chunk's projection
        _gemm(16384, 4096, 2048, name="gemm 16384x4096x2048"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "quant", "gemm", "gemm"))
    if op == "quant":
        K = 16 * _log_int(rng, 8, 512)
        return _quant(_log_int(rng, 1, min(16384, 16384 * 2048 // K)), K)
    if op == "gemm":
        K, N = 16 * _log_int(rng, 16, 256), 8 * _log_int(rng, 32, 1024)
        return _gemm(_log_int(rng, 1, min(16384, 16384 * 4096 * 2048 // (N * K))), N, K)
    D = rng.choice((64, 128, 128, 256))
    n_kv = _log_int(rng, 1, 8)
    n_q = n_kv * rng.choice((1, 2, 4, 5, 7, 8, 16))
    page, cache, heads_first = rng.choice((8, 16, 32, 64, 128)), rng.choice(("bf16", "bf16", "e4m3")), rng.random() < 0.5
    if op == "append":
        T = _log_int(rng, 1, min(16384, 16384 * 20 * 256 // ((n_q + 2 * n_kv) * D)))
        return _append(T, _log_int(rng, 1, min(T, 256)), n_q, n_kv, D, 16 * rng.randint(1, D // 16), page,
                       past=_log_int(rng, 1, 200000) - 1, cache=cache, norm=rng.random() < 0.6,
                       interleaved=rng.random() < 0.3, heads_first=heads_first)
    S = _log_int(rng, 1, 256)
    row = n_kv * D * (4 if cache == "bf16" else 2)  # bytes a cached token holds; half of L is the mean of many
    L = _log_int(rng, 1, min(300000, max(1, 2 ** 30 // (row * S))))
    new = rng.choice((1, 1, 1, 2, 3, 4, 8))
    return _attend(S, L, n_q, n_kv, D, page, new=new, idle=rng.choice((0, 0, S // 20)),
                   window=rng.choice((0, 0, _log_int(rng, 1, 4096))), cache=cache, heads_first=heads_first)


def work(case):
    c = case
    if c["op"] == "quant":
        return {"bytes": c["T"] * (3 * c["K"] + 4 * _blocks(c["K"])), "flops": 3 * c["T"] * c["K"]}
    if c["op"] == "gemm":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": T * K + N * K + 2 * T * N + 4 * _blocks(K) * (T + _blocks(N)), "flops": 2 * T * N * K}
    new, lens = _lengths(c)
    D, each = c["D"], 2 if c["cache"] == "bf16" else 1
    tables = 4 * (2 * c["S"] + 1)
    if c["op"] == "append":
        pages = sum((l - 1) // c["page"] - (l - n) // c["page"] + 1 for n, l in zip(new, lens))
        rows = c["T"] * D
        return {"bytes": rows * (4 * c["n_q"] + c["n_kv"] * (4 + 2 * each)) + 4 * pages + tables,
                "flops": rows * (c["n_q"] + c["n_kv"]) * 3}
    seen = [_seen(c, n, l) for n, l in zip(new, lens)]
    at = sum(min(l - n + 1 + i, c["window"] or l) for n, l in zip(new, lens) if l for i in range(n))
    return {"bytes": sum(seen) * c["n_kv"] * D * 2 * each + sum(new) * c["n_q"] * D * 4 + sum(v // c["page"] + 1 for v in seen) * 4 + tables,
            "flops": 4 * at * c["n_q"] * D}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _blocks(n):
    return (n + 127) // 128


def _seen(c, n, l):
    """Cached tokens that the n new ones of a request of l see together."""
    return min(l, c["window"] + n - 1) if c["window"] else l


def _lengths(c):
    """(new tokens, tokens in the cache with them) of each request. They go by the case alone; a seed does not move them."""
    S = c["S"]
    rng = random.Random(c.get("T", c.get("L")) * 1009 + S)
    if c["op"] == "append":  # half of the requests hold one token (decode steps), the rest share what is left unevenly
        T = c["T"]
        ones = S // 2 if S < T else S
        share = [rng.random() ** 2 + 0.02 for _ in range(S - ones)]
        left = T - ones - len(share)
        new = [1 + int(left * v / sum(share)) for v in share]
        if new:
            new[0] += T - ones - sum(new)
        new = [1] * ones + new
        rng.shuffle(new)
        return new, [n + (c["past"] if S == 1 else int(c["past"] * rng.random())) for n in new]
    new = [rng.randint(1, c["new"]) if S > 1 else c["new"] for _ in range(S)]
    lens = [max(n, c["L"] if S == 1 else int(c["L"] * rng.random()) + 1) for n in new]
    for i in rng.sample(range(S), min(c["idle"], S - 1)):  # a slot without a request: one row, nothing to see
        new[i], lens[i] = 1, 0
    return new, lens


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _tensor(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * std + mean

    bf = torch.bfloat16
    s = dict(c)
    if c["op"] == "quant":
        s["x"] = normal(c["T"], c["K"]).to(bf)
        s["out"] = (torch.empty(c["T"], c["K"], dtype=E4M3, device="cuda"), torch.empty(c["T"], _blocks(c["K"]), device="cuda"))
        return s
    if c["op"] == "gemm":
        T, N, K = c["T"], c["N"], c["K"]
        s["a"] = normal(T, K, std=120.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
        s["a_scale"] = normal(T, _blocks(K)).abs() * 0.002 + 0.006
        s["b"] = normal(N, K, std=120.0).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)
        s["b_scale"] = normal(_blocks(N), _blocks(K)).abs() * 0.0001 + 0.0001
        s["out"] = torch.empty(T, N, dtype=bf, device="cuda")
        return s

    new, lens = _lengths(c)
    S, D, n_q, n_kv, page, T = c["S"], c["D"], c["n_q"], c["n_kv"], c["page"], sum(new)
    rng = random.Random(int(seed))
    first = [l - n for n, l in zip(new, lens)] if c["op"] == "append" else [0] * S
    tables, used = [], 1  # page 0: what append's table names for tokens that were written earlier (it does not touch them)
    for f, l in zip(first, lens):
        head, count = f // page, (l + page - 1) // page
        tables.append([0] * head + list(range(used, used + count - head)))
        used += max(0, count - head)
    order = list(range(1, used))
    rng.shuffle(order)
    order = [0] + order
    width = max(1, max(map(len, tables)))
    s["pages"] = _tensor([[order[i] for i in t] + [0] * (width - len(t)) for t in tables])
    s["kv_len"] = _tensor(lens)
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    s["offsets"] = _tensor(off)
    s["most"] = max(new)

    def cache():
        shape = (used, n_kv, page, D) if c["heads_first"] else (used, page, n_kv, D)
        v = torch.empty(shape, dtype=bf if c["cache"] == "bf16" else E4M3, device="cuda")
        flat = v.view(-1)
        for at in range(0, flat.numel(), 1 << 28):  # what is not written yet holds earlier requests' values
            part = flat[at: at + (1 << 28)]
            v_part = normal(part.numel(), std=1.0 if c["cache"] == "bf16" else 60.0)
            part.copy_(v_part.clamp_(-E4M3_MAX, E4M3_MAX))
        return v.transpose(1, 2) if c["heads_first"] else v

    s["k_cache"], s["v_cache"] = cache(), cache()
    s["k_scale"] = s["v_scale"] = None
    if c["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = (normal(n_kv).abs() * 0.002 + 0.015 for _ in range(2))
    if c["op"] == "append":
        qkv = normal(T, (n_q + 2 * n_kv) * D, std=1.5).to(bf)  # the projection's output: q, k and v side by side
        s["q"], s["k"], s["v"] = (p.view(T, -1, D) for p in qkv.split((n_q * D, n_kv * D, n_kv * D), 1))
        s["w_q"], s["w_k"] = (normal(D, std=0.1, mean=1.0).to(bf) if c["norm"] else None for _ in range(2))
        s["inv_freq"] = 1e6 ** (-torch.arange(0, c["rot"], 2, device="cuda").float() / c["rot"])
        s["out"] = torch.empty(T, n_q, D, dtype=bf, device="cuda")
    else:
        s["q"] = normal(T, n_q, D, std=2.0).to(bf)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(T, n_q, D, dtype=bf, device="cuda")
        s["lse"] = torch.empty(T, n_q, device="cuda")
        s["width"] = max(_seen(c, n, l) for n, l in zip(new, lens))  # what a program that pads knows of its batch
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _plain_quant(s):
    x = s["x"].float()
    T, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128)).view(T, -1, 128)
    most = x.abs().amax(2)
    scale = torch.where(most == 0, 1.0, most / torch.full_like(most, E4M3_MAX))  # (by a number, torch multiplies by its reciprocal)
    codes = (x / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return codes.view(T, -1)[:, :K].to(E4M3), scale


def _plain_gemm(s):
    T, K = s["a"].shape
    N = s["b"].shape[0]
    a = s["a"].float() * s["a_scale"].repeat_interleave(128, 1)[:, :K]
    b = s["b"].float() * s["b_scale"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return (a @ b.T).to(torch.bfloat16)


def _requests(s):
    """(request, position) of each token."""
    off = s["offsets"].long()
    T = s["q"].shape[0]
    request = torch.arange(s["S"], device="cuda").repeat_interleave(off[1:] - off[:-1], output_size=T)
    return request, s["kv_len"].long()[request] - off[request + 1] + torch.arange(T, device="cuda")


def _plain_append(s):
    rot, half = s["rot"], s["rot"] // 2
    request, pos = _requests(s)
    angle = pos.double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * w.float()
        if s["interleaved"]:
            a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), 3).flatten(2)
        else:
            a, b = x[:, :, :half], x[:, :, half:rot]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), 2)
        return torch.cat((r, x[:, :, rot:]), 2)

    def held(x, scale):
        if scale is None:
            return x.to(torch.bfloat16)
        return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)

    page, slot = s["pages"][request, pos // s["page"]].long(), pos % s["page"]
    for cache, x, scale in ((s["k_cache"], turned(s["k"], s["w_k"]), s["k_scale"]), (s["v_cache"], s["v"].float(), s["v_scale"])):
        x = held(x, scale)
        if x.dtype == E4M3:  # (rows are put in place as bytes)
            cache, x = cache.view(torch.uint8), x.view(torch.uint8)
        cache[page, slot] = x
    return turned(s["q"], s["w_q"]).to(torch.bfloat16), s["k_cache"], s["v_cache"]


def _plain_attend(s):
    # the requests padded to the longest: their tokens gathered from the pages, then products over all
    S, n_q, n_kv, D, most, width, page = s["S"], s["n_q"], s["n_kv"], s["D"], s["most"], s["width"], s["page"]
    request, pos = _requests(s)
    off, lens = s["offsets"].long(), s["kv_len"].long()
    i = torch.arange(most, device="cuda")
    new = off[1:] - off[:-1]
    mine = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)              # [S, most]: the padded rows
    at = lens[:, None] - new[:, None] + i                                   # their positions
    first = (lens - new - s["window"] + 1).clamp(min=0) if s["window"] else torch.zeros_like(lens)
    there = first[:, None] + torch.arange(width, device="cuda")             # [S, width]: positions in the cache
    live = there < lens[:, None]
    there = torch.where(live, there, 0)
    which, slot = s["pages"].gather(1, there // page).long(), there % page

    def rows(cache, scale):
        if cache.dtype == E4M3:
            x = cache.view(torch.uint8)[which, slot].view(E4M3).float() * scale[:, None]
        else:
            x = cache[which, slot].float()
        return torch.where(live[:, :, None, None], x, 0.0).permute(0, 2, 3, 1)      # [S, n_kv, D, width]

    q = s["q"].float()[mine].view(S, most, n_kv, n_q // n_kv, D).permute(0, 2, 1, 3, 4).reshape(S, n_kv, -1, D)
    score = (q @ rows(s["k_cache"], s["k_scale"])) * s["scale"]
    seen = live[:, None] & (there[:, None] <= at[:, :, None])                       # [S, most, width]
    if s["window"]:
        seen = seen & (there[:, None] > at[:, :, None] - s["window"])
    seen = seen.repeat_interleave(n_q // n_kv, 1)[:, None]
    score = torch.where(seen, score, float("-inf"))
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    total = p.sum(3, keepdim=True)
    out = (p @ rows(s["v_cache"], s["v_scale"]).transpose(2, 3)) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, float("-inf"), top + torch.log(total))
    part = torch.arange(pos.numel(), device="cuda") - off[request]                  # a token's place in its request

    def back(x):
        return x.view(S, n_kv, most, n_q // n_kv, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)[request, part]

    return back(out).to(torch.bfloat16), back(lse).squeeze(2)


def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "quant": _plain_quant, "gemm": _plain_gemm}[s["op"]](s)
    import nvfp4_w4a4_mixture_gb300 as m

    if s["op"] == "quant":
        return m.moe_quantize_fp8(s["x"], out=s["out"])
    if s["op"] == "gemm":
        return m.moe_gemm_fp8(s["a"], s["a_scale"], s["b"], s["b_scale"], out=s["out"])
    if s["op"] == "append":
        q = m.moe_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["offsets"], s["kv_len"], s["pages"],
                               inv_freq=s["inv_freq"], interleaved=s["interleaved"], w_q=s["w_q"], w_k=s["w_k"], eps=EPS,
                               k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        return q, s["k_cache"], s["v_cache"]
    out = m.moe_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["offsets"], s["kv_len"], s["pages"], max_new=s["most"],
                                scale=s["scale"], window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                out=s["out"], lse=s["lse"])
    return out, s["lse"]


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_quant(s):
    # the scale is a 32-bit number and the quotient is one before it is an 8-bit one: both belong to the format
    codes = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    scales = torch.empty(s["T"], _blocks(s["K"]), dtype=torch.float64, device="cuda")
    for b in range(_blocks(s["K"])):
        x = s["x"][:, 128 * b: 128 * (b + 1)].double()
        most = x.abs().max(1).values
        f = torch.where(most > 0, most / 448, 1.0).float().double()
        q = (x / f[:, None]).float().double()
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)  # four significant bits, 2^-9 the least
        codes[:, 128 * b: 128 * (b + 1)] = (torch.round(q / step) * step).clamp(-448, 448)
        scales[:, b] = f
    return codes, scales


def _exact_gemm(s):
    out = torch.zeros(s["T"], s["N"], dtype=torch.float64, device="cuda")
    row = torch.arange(s["N"], device="cuda") // 128
    for b in range(_blocks(s["K"])):
        k = slice(128 * b, 128 * (b + 1))
        out += s["a_scale"][:, b, None].double() * (s["a"][:, k].double() @ s["b"][:, k].double().T) * s["b_scale"][row, b].double()
    return out


def _exact_append(s):
    off, lens = s["offsets"].tolist(), s["kv_len"].tolist()
    pos = torch.cat([torch.arange(l - (off[i + 1] - off[i]), l) for i, l in enumerate(lens)]).cuda()
    request = torch.cat([torch.full((off[i + 1] - off[i],), i) for i in range(len(lens))]).cuda()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None].double() * s["inv_freq"].double()[None])

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w.double()
        x = x.clone()
        r = s["rot"]
        first, second = (slice(0, r, 2), slice(1, r, 2)) if s["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    caches = []
    for cache, x, scale in (("k_cache", rotated(s["k"], s["w_k"]), s["k_scale"]), ("v_cache", s["v"].double(), s["v_scale"])):
        new = s[cache].double()
        if scale is not None:
            x = (x / scale.double()[:, None]).clamp(-448, 448)
        new[s["pages"].long()[request, torch.div(pos, s["page"], rounding_mode="floor")], torch.remainder(pos, s["page"])] = x
        caches.append(new)
    return rotated(s["q"], s["w_q"]), caches[0], caches[1]


def _exact_attend(s):
    off, lens, W = s["offsets"].tolist(), s["kv_len"].tolist(), s["window"]
    T, n_q, D = s["q"].shape
    group = n_q // s["n_kv"]
    out = torch.zeros(T, n_q, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, n_q), float("-inf"), dtype=torch.float64, device="cuda")
    for i, l in enumerate(lens):
        n = off[i + 1] - off[i]
        lo = max(0, l - n - W + 1) if W else 0
        if l == lo:
            continue
        pos = torch.arange(lo, l, device="cuda")
        page = s["pages"][i, pos // s["page"]].long()
        for h in range(s["n_kv"]):
            k, v = (s[c][page, pos % s["page"], h].double() for c in ("k_cache", "v_cache"))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for j in range(n):
                a = l - n + j
                rows = slice(max(0, a - W + 1) - lo if W else 0, a + 1 - lo)
                t, heads = off[i] + j, slice(h * group, (h + 1) * group)
                z = s["q"][t, heads].double() @ k[rows].T * s["scale"]
                lse[t, heads] = torch.logsumexp(z, 1)
                out[t, heads] = torch.softmax(z, 1) @ v[rows]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "quant": _exact_quant, "gemm": _exact_gemm}[case["op"]](s)
