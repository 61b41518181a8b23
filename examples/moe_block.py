"""A stack of mixture-of-experts blocks as a server runs it: the norm before a block, routing by sigmoid scores with a
balance bias and expert groups, the NVFP4 experts, the requests' low-rank adapters beside the block, and after it the
norm, the gate and the residual sum, which the next block's norm shares a launch with.

    python examples/moe_block.py [--tokens 2048] [--layers 4] [--requests 16]

Weights are random; the program prints the time of a pass and checks its first block against plain torch operations.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_w4a4_mixture_gb300 as m  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """One block's weights. The experts' matrices are quantised to NVFP4 on the device."""

    def __init__(self, gen, H, E, k, I, n_group, topk_group, adapters, rank, s_mid=0.002):
        def normal(*shape, std, mean=0.0):
            return torch.randn(*shape, generator=gen, device="cuda") * std + mean

        def bank(rows, cols, parts):
            codes, sf, scale = [], [], []
            for _ in range(E + 1):
                q = [m.moe_quantize_nvfp4(normal(rows // parts, cols, std=0.02)) for _ in range(parts)]
                codes.append(torch.cat([c for c, _, _ in q]))
                sf.append(torch.cat([s for _, s, _ in q]))
                scale.append(torch.cat([s for _, _, s in q]))
            scale = torch.stack(scale)
            return torch.stack(codes), torch.stack(sf), scale if parts > 1 else scale.flatten()

        self.layer = m.MoeLayer(H, E, k, I, normal(E + 1, H, std=0.02).to(BF16), bank(2 * I, H, 2), bank(H, I, 1),
                                torch.full((E + 1,), s_mid, device="cuda"))
        self.n_group, self.topk_group = n_group, topk_group
        self.bias = normal(E, std=0.02)                 # moved by the training's balance rule, for the choice alone
        self.w_pre = normal(H, std=0.1, mean=1.0).to(BF16)
        self.w_post = normal(H, std=0.1, mean=1.0).to(BF16)
        self.gate = normal(H, std=0.1, mean=0.5).to(BF16)
        self.a = normal(adapters, rank, H, std=0.02).to(BF16)
        self.b = normal(adapters, H, rank, std=0.02).to(BF16)
        self.scale = torch.full((adapters,), 2.0, device="cuda")


def experts(block, x, ids, w, shared_g):
    """The layer's experts for a routing that is given: permutation, W4A4 encoding, both expert GEMMs, combination."""
    L = block.layer
    T, k = ids.shape
    offsets, _, src_perm, row_token = m.moe_permute(ids, L.E)
    codes, sf, s = m.moe_quantize_nvfp4(x)
    rows = T * k + T
    h, h_sf = m.moe_grouped_gemm_nvfp4(codes, sf, s, offsets, rows, L.gu_codes, L.gu_sf, L.gu_scale, 2 * L.I, L.H, True,
                                       m.EPI_SWIGLU_NVFP4, a_row_index=row_token, epi_scale=L.s_mid)
    y = m.moe_grouped_gemm_nvfp4(h, h_sf, L.s_mid, offsets, rows, L.dn_codes, L.dn_sf, L.dn_scale, L.H, L.I, False, m.EPI_BF16)
    return m.moe_combine(y, w, src_perm, shared_g=shared_g)


def route(block, x):
    """(ids, weights, shared gate) of the tokens."""
    _, _, shared_g, logits = m.moe_route_topk(x, block.layer, want_logits=True)
    ids, w = m.moe_select_experts(logits, block.layer.k, bias=block.bias, score=m.SCORE_SIGMOID, n_group=block.n_group,
                                  topk_group=block.topk_group, group_score=m.GROUP_TOP2, scale=2.5)
    return ids, w, shared_g


def block_output(block, x, seg_offsets, seg_adapter):
    """The block's output of normed tokens x: experts, then each request's adapter in place."""
    y = experts(block, x, *route(block, x))
    return m.moe_adapter_add(x, y, block.a, block.b, block.scale, seg_offsets, seg_adapter, out=y)


def stack_forward(blocks, residual, seg_offsets, seg_adapter):
    """The residual stream (fp32 or bf16 [T, H]) after all blocks."""
    _, x = m.moe_norm_residual(None, residual, w_pre=blocks[0].w_pre)
    for i, block in enumerate(blocks):
        y = block_output(block, x, seg_offsets, seg_adapter)
        w_pre = blocks[i + 1].w_pre if i + 1 < len(blocks) else None
        residual, x = m.moe_norm_residual(y, residual, w_post=block.w_post, w_pre=w_pre, gate=block.gate)
    return residual


def plain_block(block, residual, seg_offsets, seg_adapter, w_next, eps=1e-6):
    """One block with the norms, the selection and the adapters in plain torch operations of 64 bits; the experts are
    the library's. Returns (residual, the next block's x)."""
    def rms(v, w):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * w.double()

    L = block.layer
    x = rms(residual.double(), block.w_pre).to(BF16)
    _, _, shared_g, logits = m.moe_route_topk(x, L, want_logits=True)
    s = torch.sigmoid(logits.double())
    c = s + block.bias.double()
    v = c.view(-1, block.n_group, L.E // block.n_group).topk(2, dim=2).values.sum(2)
    keep = torch.zeros_like(v, dtype=torch.bool).scatter(1, v.topk(block.topk_group, dim=1).indices, True)
    c = torch.where(keep.repeat_interleave(L.E // block.n_group, 1), c, float("-inf"))
    ids = c.topk(L.k, dim=1).indices
    w = s.gather(1, ids)
    w = 2.5 * w / w.sum(1, keepdim=True)
    y = experts(block, x, ids.int(), w.float(), shared_g).double()
    off = seg_offsets.tolist()
    for i, a in enumerate(seg_adapter.tolist()):
        if a >= 0:
            rows = slice(off[i], off[i + 1])
            y[rows] += float(block.scale[a]) * (x[rows].double() @ block.a[a].double().T) @ block.b[a].double().T
    residual = residual.double() + block.gate.double() * rms(y, block.w_post)
    return residual, rms(residual, w_next)


def requests_of(tokens, n, adapters, device="cuda"):
    """Offsets and adapters of n requests: ragged lengths, every fourth request on the base model alone."""
    cuts = sorted({0, tokens, *(int(tokens * (i / n) ** 1.5) for i in range(1, n))})
    ids = [-1 if i % 4 == 3 else i % adapters for i in range(len(cuts) - 1)]
    return torch.tensor(cuts, dtype=torch.int32, device=device), torch.tensor(ids, dtype=torch.int32, device=device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--intermediate", type=int, default=768)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    blocks = [Block(gen, a.hidden, a.experts, 8, a.intermediate, 8, 4, adapters=4, rank=16) for _ in range(a.layers)]
    residual = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda")
    off, ids = requests_of(a.tokens, a.requests, 4)

    ref, _ = plain_block(blocks[0], residual, off, ids, blocks[0].w_pre)
    got = stack_forward(blocks[:1], residual, off, ids)
    m.moe_read_device_status()
    print("first block against plain operations: relative error %.2e" % float((got - ref).norm() / ref.norm()))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        stack_forward(blocks, residual, off, ids)
    start.record()
    for _ in range(10):
        stack_forward(blocks, residual, off, ids)
    end.record()
    torch.cuda.synchronize()
    print("%d blocks, %d tokens: %.1f us a pass" % (a.layers, a.tokens, start.elapsed_time(end) / 10 * 1e3))


if __name__ == "__main__":
    main()
