"""mx_kv_append's queries where a head's elements, its weights and rope_scale are far from 1, and far from
each other: what is representable comes out right, whatever the terms between would be."""
import numpy as np
import pytest

import workloads as W
from oracle import mx_oracle as O
from oracle import mx_step_oracle as S

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_step import dev

pytestmark = pytest.mark.gpu


def _check(mx, x, weight, eps, rot, pairs=False, rope_scale=1.0):
    """x: values [T, H, D], rounded to bf16 here."""
    bits = W.f32_to_bf16_bits(np.asarray(x, dtype=np.float32))
    T, H, D = bits.shape
    pos = np.arange(T, dtype=np.int32) * 37
    freq = (10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
    weight = np.asarray(weight, dtype=np.float32)
    got = mx.mx_kv_append(dev_bf16(bits), None, None, dev(pos), None, None, 16, inv_freq=dev(freq) if rot else None, q_weight=dev(weight),
                          eps=eps, rope=mx.MX_ROPE_PAIRS if pairs else mx.MX_ROPE_HALVES, rope_scale=rope_scale)
    y, size = S.norm_rotate(O.bf16_to_f64(bits), pos, weight, eps, freq, pairs, rope_scale)
    assert np.abs(y).max() < 3.3e38, "the inputs are meant to have results in bf16's range"
    err, bound = np.abs(O.bf16_to_f64(host_bits(got)) - y), S.query_bound(y, size)
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, (len(bad), bad[0], y[tuple(bad[0])], err[tuple(bad[0])], bound[tuple(bad[0])])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("large,weight", [(5e17, 1e21), (-5e17, 1e38), (1.0, 1e38), (1e17, -3e36), (2e15, 1e24), (3e38, 1e37), (3e-20, 1e30)])
def test_weights_far_above_one(D, large, weight):
    """Sums of squares on both sides of where they leave FP32, times weights that would."""
    torch_or_skip()
    mx = lib_or_fail()
    x = np.full((7, 5, D), large)
    x[1::2, :, ::3] *= 2.0 ** -20
    for rot in (0, D // 2, D):
        for pairs in (False, True):
            _check(mx, x, np.full(D, weight), 0.0, rot, pairs)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-12])
def test_products_below_the_normal_numbers(D, eps):
    """Elements near the least normal number times weights below 1, and elements far below the head's others."""
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(D)
    near = rng.standard_normal((9, 5, D)) * 2.0 ** -125
    for rot in (0, D):
        for pairs in (False, True):
            for w in (1.0, 2.0 ** -10, 2.0 ** -40):
                _check(mx, near, w * (1 + rng.random(D)), eps, rot, pairs)
            mixed = rng.standard_normal((9, 5, D)) * 2.0 ** rng.integers(-120, -49, (9, 5, D)).astype(np.float64)
            _check(mx, mixed, 1 + rng.random(D), eps, rot, pairs)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("std", [1e-35, 1e-18, 1e-9, 1.0, 1e9, 1e18, 1e30, 6e37])
def test_weights_and_elements_of_every_size(D, std):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(D)
    T, H = 11, 9
    for low, high in ((-100, 100), (-100, 0), (0, 110)):
        weight = 2.0 ** rng.uniform(low, high, D) * rng.choice([-1, 1], D)
        for rot, pairs, scale in ((0, False, 1.0), (D, False, 0.5), (D, True, 2.0 ** 9), (D // 2, False, 2.0 ** -30)):
            x = rng.standard_normal((T, H, D)) * std
            x[3] *= 2.0 ** rng.integers(-20, 1, (H, D)).astype(np.float64)
            _check(mx, x, weight, 0.0 if D == 128 else 1e-6, rot, pairs, scale)
