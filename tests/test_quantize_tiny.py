"""GPU: FP8 encoding of blocks whose largest value is tiny (the scale, or its reciprocal, leaves FP32's normal numbers), with
zeros beside it, against the FP32 quotient bit for bit."""
import numpy as np
import pytest
import torch

from test_attention_ops import BF, E4M3, m  # noqa: F401

pytestmark = pytest.mark.gpu

# bits of a block's largest value: 2^-133 (the least), others without a normal number, 2^-126, 2^-118 (the scale has no normal
# number), 1.75 x 2^-118 = 448 x 2^-126 and its neighbours, 2^-117, 2^-100 and its neighbours
TOPS = [0x0001, 0x0002, 0x0003, 0x0047, 0x007F, 0x0080, 0x0081, 0x0400, 0x0401, 0x045F, 0x0460, 0x0461, 0x0480, 0x0481, 0x0D7F, 0x0D80, 0x0D81]


def encoded(x):
    """Codes and scales in NumPy's FP32, which keeps numbers below the normal ones."""
    T, K = x.shape
    p = np.zeros((T, -(-K // 128) * 128), np.float32)
    p[:, :K] = x.float().cpu().numpy()
    p = p.reshape(T, -1, 128)
    most = np.abs(p).max(2)
    scale = np.where(most == 0, np.float32(1), most / np.float32(448))
    q = np.clip(p / scale[:, :, None], -448, 448).reshape(T, -1)[:, :K]
    return torch.from_numpy(np.ascontiguousarray(q)).to(E4M3), torch.from_numpy(scale)


@pytest.mark.parametrize("T,K", [(1, 128), (34, 144), (50, 2064), (20000, 272)])  # the last: the kernel for many blocks
def test_tiny_blocks_are_exact(m, T, K):  # noqa: F811
    rng = np.random.default_rng(T)
    blocks = -(-K // 128)
    top = np.array(TOPS, np.int64)[(np.arange(T)[:, None] * blocks + np.arange(blocks)) % len(TOPS)].repeat(128, 1)[:, :K]
    bits = (rng.random((T, K)) * (top + 1)).astype(np.int64)
    bits[rng.random((T, K)) < 0.3] = 0
    pairs = rng.random((T, K // 2)) < 0.3
    bits[np.repeat(pairs, 2, 1)] = 0
    bits[:, ::128] = top[:, ::128]
    bits[:, 2:4] = 0
    bits |= (rng.random((T, K)) < 0.5).astype(np.int64) << 15
    x = torch.from_numpy(bits.astype(np.uint16).view(np.int16)).cuda().view(BF)
    codes, scale = m.moe_quantize_fp8(x)
    ref, ref_scale = encoded(x)
    assert torch.equal(scale.cpu(), ref_scale)
    assert not bool(codes.float().isnan().any())
    assert torch.equal(codes.cpu().view(torch.uint8), ref.view(torch.uint8))
