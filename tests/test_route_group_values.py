"""Group values of mx_moe_route are sums of c as they are, rounded to the bits that are compared once they are
summed: by hand for the oracle, then the kernel against it."""
import numpy as np
import pytest

from oracle import mx_step_oracle as S

from gpu_util import lib_or_fail, torch_or_skip
from test_gpu_step import _check_route

TINY = 2.0 ** -44


def _opposite(E, groups, seed, rows=12):
    """(logits, bias): in each group two experts whose c are of opposite signs and nearly the same size, the others far
    below them. The logits are odd multiples of 2^-44, another one in each group of a row, so that groups' sums differ by
    2^-45 at least, where FP64's are off by 2^-51, and that no c lies where it is cut: c has 43 bits
    below 1 and 44 below 1/2."""
    rng = np.random.default_rng(seed)
    n = E // groups
    x = np.zeros((rows, groups, n), np.float32)
    for t in range(rows):
        x[t, :, rng.integers(0, 2)] = (2 * rng.permutation(groups) + 1) * TINY
    bias = np.full((groups, n), -2.0, np.float32)
    bias[:, 0], bias[:, 1] = 0, -1
    return x.reshape(rows, E), bias.reshape(E)


def test_group_values_by_hand():
    # c = 1/2, -1/2, 1/2 + 2^-46, -1/2: sums 0 and 2^-46
    ids, _ = S.route(np.array([[0, 0, TINY, 0]]), 1, bias=[0, -1, 0, -1], sigmoid=True, groups=2, topk_groups=1)
    assert ids.tolist() == [[2]]
    ids, _ = S.route(np.array([[TINY, 0, 0, 0]]), 1, bias=[0, -1, 0, -1], sigmoid=True, groups=2, topk_groups=1)
    assert ids.tolist() == [[0]]
    # equal sums: the lower group
    ids, _ = S.route(np.zeros((1, 4)), 1, bias=[0, -1, 0, -1], sigmoid=True, groups=2, topk_groups=1)
    assert ids.tolist() == [[0]]


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,keep", [(4, 2, 1), (8, 2, 1), (64, 8, 3), (96, 6, 2), (160, 5, 1), (256, 32, 7), (1000, 50, 3), (1008, 63, 8)])
@pytest.mark.parametrize("f32", [False, True])
def test_group_values_that_cancel(E, groups, keep, f32):
    torch_or_skip()
    mx = lib_or_fail()
    x, bias = _opposite(E, groups, E)
    for topk in (1, keep):
        _check_route(mx, x, topk, f32, bias=bias, sigmoid=True, groups=groups, topk_groups=keep)
        _check_route(mx, x, topk, f32, bias=bias, sigmoid=True, groups=groups, topk_groups=keep, group_top=1)
    if E & (E - 1) == 0 and E <= 64:  # softmax of nearly equal logits: p = 1 / E times 1 + k 2^-44
        bias = np.where(bias == -1, -2.0 / E, bias).astype(np.float32)
        _check_route(mx, x, keep, f32, bias=bias, groups=groups, topk_groups=keep)


