"""GPU: groups whose values lie nearer to one another than the FP32 sums of their two largest scores are exact: the
error bound has to send them to the FP64 decision."""
import pytest
import torch

from test_block_ops import check_select, moe  # noqa: F401

pytestmark = pytest.mark.gpu

# (a1, a2, b1, b2): exp(a1) + exp(a2) is the smaller sum by 1e-9 to 7e-9, and the larger by 3.6e-7 where the terms are
# 2^(x log2 e) by the hardware's FP32 approximation (searched for; the sums are near 1, where FP32 steps are 1.2e-7)
NEAR_PAIRS = [(-0.61044842, -0.611714721, -0.363848448, -0.940248609), (-0.573789477, -0.649609804, -0.364275724, -0.939210534),
              (-0.540978014, -0.685329914, -0.36315915, -0.94000262), (-0.54147172, -0.684316874, -0.363324493, -0.939136744),
              (-0.541459322, -0.684369922, -0.36315915, -0.939480901), (-0.606469214, -0.613909364, -0.36315915, -0.938976526),
              (-0.613495469, -0.606262326, -0.36315915, -0.938115358), (-0.606456339, -0.61149013, -0.361682892, -0.938233852)]


@pytest.mark.parametrize("T,E", [(16, 1024), (16, 512), (2600, 256), (12000, 512)])
@pytest.mark.parametrize("renorm", [False, True])
def test_groups_without_bias_nearer_than_their_scores_errors(moe, T, E, renorm):  # noqa: F811
    # four groups, one far ahead; the pairs contend for the second place
    n = len(NEAR_PAIRS)
    l = (-0.96 - 1e-4 * torch.arange(E, device="cuda")).view(1, 4, E // 4).repeat(2 * n, 1, 1)
    l[:, 0, 3] = l[:, 0, 5] = 0.0
    pairs = torch.tensor(NEAR_PAIRS, device="cuda")
    for flip in (0, 1):
        l[flip * n: (flip + 1) * n, 1 + flip, 7:9] = pairs[:, :2]
        l[flip * n: (flip + 1) * n, 2 - flip, 10:12] = pairs[:, 2:]
    l = l.reshape(2 * n, E).repeat((T + 2 * n - 1) // (2 * n), 1)[:T]
    check_select(moe, l, 4, score="softmax", G=4, keep=2, top2=True, renorm=renorm)
