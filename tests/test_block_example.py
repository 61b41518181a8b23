"""GPU: the example's block (norms, score routing, NVFP4 experts, adapters) against one whose norms, selection and
adapters are plain torch operations in 64 bits. A bf16 x that rounds the other way moves a token's NVFP4 codes, so the
bar is the layer's own: 2e-2 relative Frobenius error of what the block adds to the residual stream."""
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
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,requests,res", [(1, 1, torch.float32), (4, 2, torch.bfloat16), (130, 9, torch.float32),
                                                 (700, 40, torch.bfloat16)])
def test_block_matches_plain_operations(ex, tokens, requests, res):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    block = ex.Block(gen, 256, 32, 4, 128, 8, 4, adapters=3, rank=8)
    residual = torch.randn(tokens, 256, generator=gen, device="cuda").to(res)
    off, ids = ex.requests_of(tokens, requests, 3)
    got = ex.stack_forward([block], residual, off, ids)
    ex.m.moe_read_device_status()
    ref, _ = ex.plain_block(block, residual, off, ids, block.w_pre)
    added, want = got.double() - residual.double(), ref - residual.double()
    # a bf16 residual stream is rounded once more: half a step of its values
    slack = 2.0 ** -8 * float(ref.norm()) if res == torch.bfloat16 else 0.0
    assert float((added - want).norm()) <= 2e-2 * float(want.norm()) + slack


def test_stack_of_blocks_repeats_itself(ex):
    gen = torch.Generator(device="cuda").manual_seed(3)
    blocks = [ex.Block(gen, 256, 32, 4, 128, 8, 4, adapters=3, rank=8) for _ in range(3)]
    residual = torch.randn(200, 256, generator=gen, device="cuda")
    off, ids = ex.requests_of(200, 7, 3)
    first = ex.stack_forward(blocks, residual, off, ids)
    assert bool(first.isfinite().all()) and torch.equal(first, ex.stack_forward(blocks, residual, off, ids))
