"""GPU: groups whose values lie nearer to one another than the FP32 sums of their two largest scores are exact: the
error bound has to send them to the FP64 decision."""
import pytest
import torch

from test_block_ops import check_select, gen, moe, randn  # noqa: F401

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


@pytest.mark.parametrize("T,E,G,keep", [(4096, 512, 8, 4), (4096, 256, 8, 4), (3000, 64, 16, 3), (500, 1020, 17, 9)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("big", [1000.0, 3e7])
def test_groups_whose_biases_cancel(moe, T, E, G, keep, score, big):  # noqa: F811
    # a group's two largest values are near +big and -big: their sum is small, its FP32 rounding is not
    g = gen(T + E)
    bias = torch.full((G, E // G), -10 * big, device="cuda")
    bias[:, 0], bias[:, 1] = big, -big
    check_select(moe, randn(g, T, E), keep, bias=bias.reshape(-1), score=score, G=G, keep=keep)
    bias[1::2, 0], bias[1::2, 1] = 0.5, -0.5  # every other group's sum is nearly exact
    check_select(moe, randn(g, T, E), keep, bias=bias.reshape(-1), score=score, G=G, keep=keep)


@pytest.mark.parametrize("T,E,G", [(4096, 512, 8), (4096, 256, 8), (700, 1020, 17)])
def test_groups_whose_second_values_lie_far_below_the_first(moe, T, E, G):  # noqa: F811
    # scores near a rounding border of score - 1000: the second largest in FP32 is not always the second largest
    g = gen(T + E + 1)
    bias = torch.full((G, E // G), -1000.0, device="cuda")
    bias[:, 0] = 0.0
    l = randn(g, T, E, std=4e-7, mean=1.2207e-4).view(T, G, E // G)
    l[:, :, 0] = 1.0
    check_select(moe, l.reshape(T, E), 4, bias=bias.reshape(-1), G=G, keep=4)


def test_groups_whose_sums_leave_the_range(moe):  # noqa: F811
    # two biases whose FP32 sum is infinite: the 64-bit sums tell the groups apart
    E, G = 64, 8
    bias = torch.zeros(G, E // G, device="cuda")
    bias[2, 1], bias[2, 3] = 2e38, 2.0e38
    bias[5, 1], bias[5, 3] = 2e38, 2.5e38
    bias[6, 0], bias[6, 2] = 3e38, -3e38
    g = gen(9)
    for T in (8, 2600):
        check_select(moe, randn(g, T, E), 2, bias=bias.reshape(-1), G=G, keep=1)
