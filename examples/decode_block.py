"""A whole block of a model as a server decodes with it: the norm, the FP8 projection to queries, keys and values, their norm,
rotation and append to the paged cache, attention over it, the FP8 output projection, the residual sum with the norm before
the experts, and the mixture-of-experts half of moe_block.py.

    python examples/decode_block.py [--requests 32] [--context 1000] [--steps 20]

Weights are random. The program fills the cache window by window, checks a step's attention half against plain torch
operations, and prints the time of a step from a captured graph.
"""
import argparse
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)
import nvfp4_w4a4_mixture_gb300 as m  # noqa: E402
import moe_block  # noqa: E402

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
WINDOW = 16  # the most new tokens of a request in one call of the attention


def fp8_weight(w):
    """(codes, scales) of w [N, K]: a scale for each block of 128 x 128."""
    N, K = w.shape
    p = torch.nn.functional.pad(w, (0, -K % 128, 0, -N % 128))
    p = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    scale = (p.abs().amax((1, 3)) / 448).clamp(min=1e-12)
    return (p / scale[:, None, :, None]).view(-1, p.shape[2] * 128)[:N, :K].to(E4M3).contiguous(), scale.contiguous()


def fp8_value(codes, scale):
    """What codes with scales for blocks of 128 (of a row, or of 128 rows) stand for, in 64 bits."""
    rows = 1 if scale.shape[0] == codes.shape[0] else 128
    s = scale.double().repeat_interleave(rows, 0)[: codes.shape[0]].repeat_interleave(128, 1)[:, : codes.shape[1]]
    return codes.double() * s


class Attention:
    """The attention half's weights."""

    def __init__(self, gen, H, n_q, n_kv, D, rot, base=1e6):
        def normal(*shape, std, mean=0.0):
            return torch.randn(*shape, generator=gen, device="cuda") * std + mean

        self.n_q, self.n_kv, self.D = n_q, n_kv, D
        self.qkv = fp8_weight(normal((n_q + 2 * n_kv) * D, H, std=0.02))
        self.out = fp8_weight(normal(H, n_q * D, std=0.02))
        self.w_q, self.w_k = (normal(D, std=0.1, mean=1.0).to(BF16) for _ in range(2))
        self.w_pre = normal(H, std=0.1, mean=1.0).to(BF16)
        self.inv_freq = base ** (-torch.arange(0, rot, 2, device="cuda").float() / rot)


class Cache:
    """A paged cache for `requests` of up to `tokens` each, its pages handed out in turn."""

    def __init__(self, requests, tokens, n_kv, D, page=16, dtype=BF16):
        width = -(-tokens // page)
        shape = (requests * width, page, n_kv, D)
        self.k, self.v = (torch.zeros(shape, device="cuda").to(dtype) for _ in range(2))
        self.scales = (None, None) if dtype is BF16 else tuple(torch.full((n_kv,), 0.02, device="cuda") for _ in range(2))
        self.pages = torch.arange(requests * width, dtype=torch.int32, device="cuda").view(width, requests).T.contiguous()
        self.kv_len = torch.zeros(requests, dtype=torch.int32, device="cuda")


def attention_half(a, x, cache, offsets, max_new):
    """The attention's output for normed tokens x, which it appends to the cache (cache.kv_len counts them already)."""
    T = x.shape[0]
    qkv = m.moe_gemm_fp8(*m.moe_quantize_fp8(x), *a.qkv)
    q, k, v = (p.view(T, -1, a.D) for p in qkv.split((a.n_q * a.D, a.n_kv * a.D, a.n_kv * a.D), 1))
    ks, vs = cache.scales
    m.moe_cache_append(q, k, v, cache.k, cache.v, offsets, cache.kv_len, cache.pages, inv_freq=a.inv_freq, w_q=a.w_q, w_k=a.w_k,
                       k_scale=ks, v_scale=vs, out=q)
    o = m.moe_paged_attention(q, cache.k, cache.v, offsets, cache.kv_len, cache.pages, max_new=max_new, k_scale=ks, v_scale=vs)
    return m.moe_gemm_fp8(*m.moe_quantize_fp8(o.view(T, a.n_q * a.D)), *a.out)


def plain_attention_half(a, x, cache, offsets, eps=1e-6):
    """The same in plain torch operations of 64 bits, over the keys and values that the cache holds; what the library rounds
    to bf16 or FP8 between its calls is rounded here, too."""
    T, off, lens = x.shape[0], offsets.tolist(), cache.kv_len.tolist()
    qkv = (fp8_value(*m.moe_quantize_fp8(x)) @ fp8_value(*a.qkv).T).to(BF16)
    q = qkv[:, : a.n_q * a.D].double().view(T, a.n_q, a.D)
    q = q / torch.sqrt((q * q).mean(2, keepdim=True) + eps) * a.w_q.double()
    out = torch.zeros(T, a.n_q, a.D, dtype=torch.float64, device="cuda")
    half = a.inv_freq.numel()
    for s, n in enumerate(o - b for b, o in zip(off, off[1:])):
        p = torch.arange(lens[s], device="cuda")
        page = cache.pages[s, p // cache.k.shape[1]].long()
        k, v = (c.view(torch.uint8)[page, p % c.shape[1]].view(E4M3).double() if c.dtype is E4M3 else c[page, p % c.shape[1]].double()
                for c in (cache.k, cache.v))
        if cache.scales[0] is not None:
            k, v = k * cache.scales[0].double()[:, None], v * cache.scales[1].double()[:, None]
        for i in range(n):
            t, pos = off[s] + i, lens[s] - n + i
            angle = pos * a.inv_freq.double()
            r = q[t].clone()
            r[:, :half] = q[t, :, :half] * angle.cos() - q[t, :, half: 2 * half] * angle.sin()
            r[:, half: 2 * half] = q[t, :, :half] * angle.sin() + q[t, :, half: 2 * half] * angle.cos()
            r = r.to(BF16).double().view(a.n_kv, -1, a.D)
            z = torch.einsum("hgd,lhd->hgl", r, k[: pos + 1]) * a.D ** -0.5
            out[t] = torch.einsum("hgl,lhd->hgd", torch.softmax(z, 2), v[: pos + 1]).reshape(a.n_q, a.D)
    return fp8_value(*m.moe_quantize_fp8(out.to(BF16).view(T, -1))) @ fp8_value(*a.out).T


def block_forward(a, block, residual, cache, offsets, max_new, adapter_ids):
    """One block: the residual stream after both halves."""
    _, x = m.moe_norm_residual(None, residual, w_pre=a.w_pre)
    y = attention_half(a, x, cache, offsets, max_new)
    residual, x = m.moe_norm_residual(y, residual, w_pre=block.w_pre)
    y = moe_block.block_output(block, x, offsets, adapter_ids)
    return m.moe_norm_residual(y, residual, w_post=block.w_post, gate=block.gate)[0]


def fill(a, block, cache, context, hidden, gen, ids):
    """Runs `context` tokens of every request through the block, a window of up to 16 of each at a time."""
    S = cache.kv_len.shape[0]
    for at in range(0, context, WINDOW):
        n = min(WINDOW, context - at)
        offsets = torch.arange(0, (S + 1) * n, n, dtype=torch.int32, device="cuda")
        cache.kv_len.add_(n)
        block_forward(a, block, torch.randn(S * n, hidden, generator=gen, device="cuda"), cache, offsets, n, ids)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--context", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    args = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    a = Attention(gen, args.hidden, 16, 2, 256, 64)
    block = moe_block.Block(gen, args.hidden, args.experts, 8, 768, 8, 4, adapters=4, rank=16)
    S = args.requests
    cache = Cache(S, args.context + args.steps + 8, a.n_kv, a.D, dtype=BF16 if args.cache == "bf16" else E4M3)
    ids = torch.tensor([-1 if i % 4 == 3 else i % 4 for i in range(S)], dtype=torch.int32, device="cuda")
    fill(a, block, cache, args.context, args.hidden, gen, ids)
    offsets = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    residual = torch.randn(S, args.hidden, generator=gen, device="cuda")
    cache.kv_len.add_(1)
    _, x = m.moe_norm_residual(None, residual, w_pre=a.w_pre)
    got = attention_half(a, x, cache, offsets, 1).double()
    m.moe_read_device_status()
    ref = plain_attention_half(a, x, cache, offsets)
    print("attention half against plain operations: relative error %.2e" % float((got - ref).norm() / ref.norm()))

    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        block_forward(a, block, residual, cache, offsets, 1, ids)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        cache.kv_len.add_(1)
        block_forward(a, block, residual, cache, offsets, 1, ids)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print("%d requests over %d tokens and on: %.1f us a step of one block" % (S, args.context, start.elapsed_time(end) / args.steps * 1e3))


if __name__ == "__main__":
    main()
