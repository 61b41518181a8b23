"""Cases of the operators around the mixture-of-experts layer: the norms on both sides of a block with its gate and
residual scale, routing by scores with a balance bias and expert groups, and the low-rank adapters of many requests.

run() computes a case in plain torch operations, or with `own` through nvfp4_w4a4_mixture_gb300.
"""
import random

import numpy as np
import torch

own = False

EPS = 1e-6
GATES = ("none", "channel", "token", "element")


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _norm(T, H, res="bf16", gate="none", post=True, offset=0.0, alpha=1.0, **kw):
    return dict(op="norm", T=T, H=H, res=res, gate=gate, post=post, offset=offset, alpha=alpha, **kw)


def _route(T, E, k, score="sigmoid", bias=True, groups=1, keep=1, group_score="top2", renorm=True, scale=1.0,
           dtype="f32", **kw):
    return dict(op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, keep=keep, group_score=group_score,
                renorm=renorm, scale=scale, dtype=dtype, **kw)


def _adapt(T, S, n, r, K, N, bare=0, **kw):
    return dict(op="adapt", T=T, S=S, n=n, r=r, K=K, N=N, bare=bare, **kw)


def listed():
    return [
        # a decode step: the verify window of four tokens through the norm after a block and before the next
        _norm(4, 2048, name="norm 4x2048"),
        # the widest hidden size, FP32 residual stream, one gate per token (a gated block output)
        _norm(70, 8192, res="f32", gate="token", offset=1.0, name="norm 70x8192 f32 token gate"),
        # a long ragged prompt, a hidden size off the powers of two, a gate per element, no norm after the block
        _norm(12365, 2056, gate="element", post=False, alpha=0.5, name="norm 12365x2056 element gate"),
        # a long prefill chunk, a learned gate per channel
        _norm(16384, 2048, gate="channel", name="norm 16384x2048 channel gate"),
        # a decode step's routing: sigmoid scores and a balance bias
        _route(4, 512, 10, name="route 4x512"),
        # a prefill chunk from a router that leaves bf16 logits: softmax, ties in the logits
        _route(2048, 512, 10, score="softmax", bias=False, dtype="bf16", name="route 2048x512 softmax bf16"),
        # a long ragged prompt, groups whose size is no power of two, weights as the softmax gave them
        _route(12365, 160, 6, score="softmax", bias=False, groups=8, keep=3, group_score="max", renorm=False, scale=2.5,
               name="route 12365x160 3 of 8 groups"),
        # a long prefill chunk with groups limited to half of them
        _route(16384, 512, 10, groups=8, keep=4, scale=2.5, name="route 16384x512 4 of 8 groups"),
        # a decode step: two requests in one verify window
        _adapt(4, 2, 2, 16, 2048, 2048, name="adapt 4 tokens r16"),
        # a full decode batch: each token another request, a quarter of them on the base model alone
        _adapt(256, 256, 32, 32, 2048, 2048, bare=64, name="adapt 256 requests r32"),
        # prompts and decode steps mixed, ragged, a rank and widths off the powers of two
        _adapt(4113, 77, 12, 40, 2056, 1032, bare=5, name="adapt 4113 mixed r40"),
        # a long prefill chunk of eight adapters
        _adapt(16384, 24, 8, 64, 2048, 2048, name="adapt 16384 r64"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("norm", "route", "adapt"))
    if op == "norm":
        H, res, gate = 8 * _log_int(rng, 16, 1024), rng.choice(("bf16", "bf16", "f32")), rng.choice(GATES)
        each = (12 if res == "f32" else 8) + (2 if gate == "element" else 0)  # bytes an element moves
        return _norm(_log_int(rng, 1, min(16384, 16384 * 2048 * 8 // (each * H))), H, res=res, gate=gate,
                     post=rng.random() < 0.7, offset=rng.choice((0.0, 1.0)), alpha=rng.choice((1.0, 0.5, 0.7071)))
    if op == "route":
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 192, 256, 320, 384, 512))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 4])
        keep = rng.randint(max(1, (groups + 1) // 2), groups)
        return _route(_log_int(rng, 1, 16384), E, rng.randint(1, min(16, keep * (E // groups))),
                      score=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.6, groups=groups, keep=keep,
                      group_score=rng.choice(("max", "top2")), renorm=rng.random() < 0.7,
                      scale=rng.choice((1.0, 2.5)), dtype=rng.choice(("f32", "f32", "bf16")))
    T = _log_int(rng, 1, 16384)
    S = _log_int(rng, 1, min(T, 256))
    r = rng.choice((8, 16, 16, 24, 32, 40, 64))
    K, N = 8 * _log_int(rng, 32, 256), 8 * _log_int(rng, 32, 256)
    n = _log_int(rng, 1, max(1, min(S, 32 if T <= 2048 else 512 // r)))
    return _adapt(T, S, n, r, K, N, bare=rng.randint(0, (S - n) // 2))


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "norm":
        H, rb = c["H"], 2 if c["res"] == "bf16" else 4
        g = {"none": 0, "channel": 2 * H, "token": 4 * T, "element": 2 * T * H}[c["gate"]]
        w = 2 * H * (2 if c["post"] else 1)
        return {"bytes": T * H * (2 + rb + rb + 2) + g + w, "flops": T * H * 10}
    if c["op"] == "route":
        E = c["E"]
        return {"bytes": T * E * (4 if c["dtype"] == "f32" else 2) + (4 * E if c["bias"] else 0) + T * c["k"] * 8,
                "flops": T * E * 6}
    lens, bare = _lengths(c)
    with_adapter = T - sum(lens[:bare])
    K, N, r = c["K"], c["N"], c["r"]
    return {"bytes": 2 * (with_adapter * K + 2 * T * N) + c["n"] * (r * (K + N) * 2 + 4) + 4 * (2 * c["S"] + 1),
            "flops": 2 * with_adapter * r * (K + N)}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _lengths(c):
    """The requests' lengths of an adapter case, the `bare` ones (no adapter) first: half of the requests hold one
    token (decode steps), the rest share what is left unevenly. They go by the case alone; a seed orders them."""
    T, S = c["T"], c["S"]
    rng = random.Random(T * 1009 + S)
    if S == T:
        return [1] * S, c["bare"]
    ones = S // 2
    share = [rng.random() ** 2 + 0.02 for _ in range(S - ones)]
    left = T - ones - len(share)  # each of the others has one token at least
    lens = [1 + int(left * v / sum(share)) for v in share]
    lens[0] += T - ones - sum(lens)
    lens = [1] * ones + lens
    rng.shuffle(lens)
    return lens, c["bare"]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def prepare(case, seed):
    c, g = case, _gen(seed)
    T = c["T"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device="cuda") * std + mean

    bf = torch.bfloat16
    s = dict(c)
    if c["op"] == "norm":
        H = c["H"]
        rt = bf if c["res"] == "bf16" else torch.float32
        s["y"] = normal(T, H, std=0.5).to(bf)
        s["r"] = normal(T, H, std=2.0).to(rt)
        s["w_post"] = normal(H, std=0.1, mean=1.0 - c["offset"]).to(bf) if c["post"] else None
        s["w_pre"] = normal(H, std=0.1, mean=1.0 - c["offset"]).to(bf)
        s["g"] = {"none": lambda: None, "channel": lambda: normal(H, std=0.1, mean=0.5).to(bf),
                  "token": lambda: torch.sigmoid(normal(T, 1)),
                  "element": lambda: torch.tanh(normal(T, H)).to(bf)}[c["gate"]]()
        s["out"] = (torch.empty_like(s["r"]), torch.empty_like(s["y"]))
    elif c["op"] == "route":
        s["logits"] = normal(T, c["E"]).to(torch.float32 if c["dtype"] == "f32" else bf)
        s["b"] = normal(c["E"], std=0.02) if c["bias"] else None
        s["out"] = (torch.empty(T, c["k"], dtype=torch.int32, device="cuda"),
                    torch.empty(T, c["k"], dtype=torch.float32, device="cuda"))
    else:
        lens, bare = _lengths(c)
        n, r, K, N, S = c["n"], c["r"], c["K"], c["N"], c["S"]
        rng = random.Random(int(seed))
        ids = [-1] * bare + [i % n for i in range(S - bare)]
        order = list(range(S))
        rng.shuffle(order)
        off = np.concatenate([[0], np.cumsum([lens[i] for i in order])]).astype(np.int32)
        s["offsets"] = torch.from_numpy(off).cuda()
        s["ids"] = torch.tensor([ids[i] for i in order], dtype=torch.int32, device="cuda")
        s["x"] = normal(T, K).to(bf)
        s["y"] = normal(T, N, std=0.5).to(bf)
        s["a"] = normal(n, r, K, std=0.02).to(bf)
        s["b"] = normal(n, N, r, std=0.02).to(bf)
        s["s"] = normal(n, std=0.2, mean=2.0)
        s["out"] = torch.empty_like(s["y"])
    return s


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _plain_norm(s):
    u, r = s["y"].float(), s["r"].float()
    if s["post"]:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * (s["offset"] + s["w_post"].float())
    if s["g"] is not None:
        u = u * s["g"].float()
    r = s["alpha"] * r + u
    x = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * (s["offset"] + s["w_pre"].float())
    return r.to(s["r"].dtype), x.to(torch.bfloat16)


def _plain_route(s):
    # the choice is made in 64 bits: two experts' values can lie closer than 32 bits tell apart
    l = s["logits"].double()
    T, E, k = s["T"], s["E"], s["k"]
    if s["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.max(1, keepdim=True).values)
        p = p / p.sum(1, keepdim=True)
    c = p if s["b"] is None else p + s["b"].double()
    if s["groups"] > 1:
        v = c.view(T, s["groups"], E // s["groups"])
        v = v.sort(dim=2, descending=True).values[:, :, :2]
        v = v[:, :, 0] if s["group_score"] == "max" else v.sum(2)
        rank = v.sort(dim=1, descending=True, stable=True).indices[:, : s["keep"]]
        keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=l.device).scatter(1, rank, True)
        c = torch.where(keep.repeat_interleave(E // s["groups"], 1), c, float("-inf"))
    ids = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), (w * s["scale"]).float()


def _plain_adapt(s):
    # every token through every adapter of the batch as one product, then its own adapter's part alone
    T, n, r = s["T"], s["n"], s["r"]
    lens = s["offsets"][1:] - s["offsets"][:-1]
    mine = s["ids"].repeat_interleave(lens, output_size=T)
    h = s["x"].float() @ s["a"].float().view(n * r, -1).T
    at = torch.arange(n, device=h.device)
    h = torch.where((mine[:, None] == at)[:, :, None], h.view(T, n, r) * s["s"][:, None], 0.0)
    d = h.view(T, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    return (s["y"].float() + d).to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        return {"norm": _plain_norm, "route": _plain_route, "adapt": _plain_adapt}[s["op"]](s)
    import nvfp4_w4a4_mixture_gb300 as m

    if s["op"] == "norm":
        return m.moe_norm_residual(s["y"], s["r"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["g"],
                                   residual_scale=s["alpha"], eps=EPS, w_offset=s["offset"], out=s["out"])
    if s["op"] == "route":
        return m.moe_select_experts(s["logits"], s["k"], bias=s["b"],
                                    score=m.SCORE_SIGMOID if s["score"] == "sigmoid" else m.SCORE_SOFTMAX,
                                    n_group=s["groups"], topk_group=s["keep"],
                                    group_score=m.GROUP_MAX if s["group_score"] == "max" else m.GROUP_TOP2,
                                    renormalize=s["renorm"], scale=s["scale"], out=s["out"])
    return m.moe_adapter_add(s["x"], s["y"], s["a"], s["b"], s["s"], s["offsets"], s["ids"], out=s["out"])


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _exact_norm(s):
    def rms(v, w):
        return v / torch.sqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS) * (w.double() + s["offset"])

    u = s["y"].double()
    u = rms(u, s["w_post"]) if s["post"] else u
    r = s["r"].double() * s["alpha"] + (u if s["g"] is None else s["g"].double() * u)
    return r, rms(r, s["w_pre"])


def _exact_route(s):
    l = s["logits"].double().cpu().numpy()
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    if s["score"] == "sigmoid":
        p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    else:
        p = np.exp(l - np.log(np.exp(l).sum(1, keepdims=True)))
    c = p + (0 if s["b"] is None else s["b"].double().cpu().numpy())
    if G > 1:
        size = E // G
        top = -np.sort(-c.reshape(T, G, size), axis=2)
        v = top[:, :, 0] + (top[:, :, 1] if s["group_score"] == "top2" else 0)
        place = np.argsort(np.argsort(-v, axis=1, kind="stable"), axis=1)
        c = np.where(np.repeat(place < s["keep"], size, axis=1), c, -np.inf)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    w = w * s["scale"] / (w.sum(1, keepdims=True) if s["renorm"] else 1.0)
    return torch.from_numpy(ids.astype(np.int32)), torch.from_numpy(w)


def _exact_adapt(s):
    out = s["y"].double()
    off = s["offsets"].tolist()
    for i, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            rows = slice(off[i], off[i + 1])
            h = torch.einsum("tk,rk->tr", s["x"][rows].double(), s["a"][a].double())
            out[rows] += float(s["s"][a]) * torch.einsum("tr,nr->tn", h, s["b"][a].double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "adapt": _exact_adapt}[case["op"]](s)
