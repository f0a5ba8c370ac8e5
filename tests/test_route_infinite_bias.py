"""A bias of +inf counts as float32's largest number in mx_moe_route: by hand for the oracle, then the kernel
against it."""
import numpy as np
import pytest

from oracle import mx_step_oracle as S

from gpu_util import lib_or_fail, torch_or_skip
from test_gpu_step import _check_route

INF = np.inf


def test_infinite_biases_by_hand():
    # two of them outweigh one
    ids, _ = S.route(np.zeros((1, 4)), 2, bias=[INF, 0, INF, INF], sigmoid=True, groups=2, topk_groups=1)
    assert ids.tolist() == [[2, 3]]
    # and one equals the largest number: the lower group, the lower expert
    ids, _ = S.route(np.zeros((1, 4)), 1, bias=[0, S.FLT_MAX, 0, INF], sigmoid=True, groups=2, topk_groups=1)
    assert ids.tolist() == [[1]]
    ids, _ = S.route(np.zeros((1, 4)), 3, bias=[0, S.FLT_MAX, 0, INF])
    assert ids.tolist() == [[1, 3, 0]]


@pytest.mark.gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_infinite_biases(f32, sigmoid):
    torch_or_skip()
    mx = lib_or_fail()
    for E, groups, keep in ((4, 2, 1), (64, 8, 3), (160, 5, 2), (896, 1, 1), (1024, 2, 1)):
        rng = np.random.default_rng(E)
        x = rng.integers(-2, 3, (20, E)).astype(np.float32)
        for _ in range(4):
            bias = np.where(rng.random(E) < 0.15, INF, rng.integers(-1, 2, E) * 0.25).astype(np.float32)
            bias[rng.random(E) < 0.05] = S.FLT_MAX
            bias[rng.random(E) < 0.05] = -S.FLT_MAX
            bias[rng.random(E) < 0.05] = np.nan
            for top in (1, 2):
                _check_route(mx, x, min(4, keep * E // groups), f32, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=keep, group_top=top)
