"""GPU: the attention half as it is used, its calls one after the other (FP8 projection, norm, rotation and append, attention,
FP8 projection), against plain torch operations in 64 bits that round where the calls hand over; and a step of a whole block
from a captured graph against the same step called directly."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_w4a4_mixture_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("S,H,n_q,n_kv,D,rot", [(1, 256, 8, 2, 64, 32), (5, 384, 6, 1, 128, 128), (3, 256, 16, 2, 256, 64)])
def test_attention_half(ex, dtype, S, H, n_q, n_kv, D, rot):
    gen = torch.Generator(device="cuda").manual_seed(S)
    a = ex.Attention(gen, H, n_q, n_kv, D, rot)
    cache = ex.Cache(S, 60, n_kv, D, dtype=dtype)
    for n in (16, 9, 1, 4, 1):  # windows of a prompt, then decode steps and a verify window
        offsets = torch.arange(0, (S + 1) * n, n, dtype=torch.int32, device="cuda")
        cache.kv_len.add_(n)
        x = torch.randn(S * n, H, generator=gen, device="cuda").to(torch.bfloat16)
        got = ex.attention_half(a, x, cache, offsets, n).double()
        ex.m.moe_read_device_status()
        ref = ex.plain_attention_half(a, x, cache, offsets)
        # the output's own rounding (2^-8 at most) and where an intermediate value rounds the other way: a query's or an
        # output's bf16 step (2^-7 of it, seldom), an FP8 code of the attention's output (2^-3 of it, where it lies within
        # an error of the border: one in some hundred). The sum of independent ones stays within 2e-2 of the whole.
        assert float((got - ref).norm()) <= 2e-2 * float(ref.norm())


def test_step_from_a_graph(ex):
    gen = torch.Generator(device="cuda").manual_seed(7)
    S, H = 6, 256
    a = ex.Attention(gen, H, 8, 2, 64, 32)
    block = ex.moe_block.Block(gen, H, 32, 4, 128, 8, 4, adapters=3, rank=8)
    ids = torch.tensor([0, -1, 2, 1, -1, 0], dtype=torch.int32, device="cuda")
    cache = ex.Cache(S, 80, 2, 64)
    ex.fill(a, block, cache, 40, H, gen, ids)
    offsets = torch.arange(S + 1, dtype=torch.int32, device="cuda")
    residual = torch.randn(S, H, generator=gen, device="cuda")
    out = torch.empty(S, H, device="cuda")

    def step():
        cache.kv_len.add_(1)
        out.copy_(ex.block_forward(a, block, residual, cache, offsets, 1, ids))

    keep = cache.kv_len.clone(), cache.k.clone(), cache.v.clone()
    direct = []
    for _ in range(3):
        step()
        direct.append(out.clone())
    for t, v in zip((cache.kv_len, cache.k, cache.v), keep):
        t.copy_(v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, v in zip((cache.kv_len, cache.k, cache.v), keep):
        t.copy_(v)
    for want in direct:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
