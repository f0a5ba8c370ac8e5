"""mx_kv_attention at the ends of what it takes: the smallest and largest scales, queries down to
bf16's least subnormal, values whose sums come near FP32's end. Bounds are the oracle's."""
import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O

from gpu_util import lib_or_fail, torch_or_skip
from test_gpu_kv import Case
from test_gpu_kv_masks import plan_of

pytestmark = pytest.mark.gpu

KERNELS = [("few", 64, [1, 3], [90, 200]), ("few", 128, [1, 3], [90, 200]), ("few", 256, [1, 3], [90, 200]),
           ("many", 64, [140], [200]), ("many", 128, [140], [200]), ("many", 256, [140], [200])]


@pytest.mark.parametrize("kernel,D,q,kv", KERNELS)
@pytest.mark.parametrize("scale_exp,q_exp", [(-149, 0), (-130, 90), (-126, 60), (100, -104), (113, -116), (120, -124), (127, -128)])
def test_scales_and_queries_at_their_ends(kernel, D, q, kv, scale_exp, q_exp):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, 2, 1, 16, q, kv, seed=D + q_exp % 97)
    c.q = W.f32_to_bf16_bits((O.bf16_to_f64(c.q) * 2.0 ** q_exp).astype(np.float32))
    assert O.bf16_to_f64(c.q).any()
    assert plan_of(mx, c).startswith(f"k_kv_attn_{kernel}<{D}")
    c.check(mx, scale=2.0 ** scale_exp, what=f"scale 2^{scale_exp}, queries 2^{q_exp}")


@pytest.mark.parametrize("kernel,D,q,kv", KERNELS)
def test_values_whose_weighted_sums_stay_in_fp32(kernel, D, q, kv):
    """Each element's values add up to just under 2^128 / 2^8, which the weights at a lagging maximum
    may multiply by 2^8."""
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, 2, 1, 16, q, kv, seed=D, q_std=3.0)
    m, P = D // 32, c.page
    top = 127 + 120 - int(np.ceil(np.log2(6 * max(kv))))
    for b, L in enumerate(kv):
        for tok in range(L):
            for j in range(m):
                c.cache[c.table[b, tok // P], :, KV.byte_of("vs", P, D, tok % P, j)] = top
    assert plan_of(mx, c).startswith(f"k_kv_attn_{kernel}<{D}")
    c.check(mx, what="large values")
