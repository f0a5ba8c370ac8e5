"""What must not reach a result of mx_kv_attention: bytes of tokens that no row sees, in every
kernel the call can take. Exact values and bounds are the float64 oracle's."""
import numpy as np
import pytest

from oracle import mx_kv_oracle as KV

from gpu_util import lib_or_fail, torch_or_skip
from test_gpu_kv import Case

pytestmark = pytest.mark.gpu


def plan_of(mx, c, window=0, max_q=None, max_kv=None, workspace=None):
    """The kernels that Case.check's call launches, its hints being what it passes by default."""
    return mx.mx_kv_attention_plan(len(c.kv_lens), c.T, c.H * c.G, c.H, c.D, max_q or max(c.q_lens + [1]),
                                   max_kv or max(c.kv_lens + [1]), window, workspace_bytes=0 if workspace is False else None)


def fill_tokens(c, b, tokens, codes, scales):
    """Bytes of request b's tokens, in every head: codes and scales are a byte or arrays of them."""
    mk, mv, mks, mvs = KV._maps(c.page, c.D)
    for tok in tokens:
        blk = c.cache[c.table[b, tok // c.page]]
        for maps, to in (((mk, mv), codes), ((mks, mvs), scales)):
            for m in maps:
                at = m[tok % c.page].reshape(-1)
                blk[:, at] = to if np.isscalar(to) else to(len(blk), at.size)


# D, H, G, page, q, kv, window, workspace, what the plan names
WINDOWS = [
    (64, 2, 3, 16, [1, 4], [200, 90], 37, None, ["k_kv_attn_few<64, 1, false>"]),
    (64, 1, 8, 16, [4, 4], [200, 90], 38, None, ["k_kv_attn_few<64, 2, false>"]),
    (128, 2, 3, 32, [1, 4], [200, 90], 21, None, ["k_kv_attn_few<128, 1, false>"]),
    (128, 1, 8, 32, [4, 4], [200, 90], 23, None, ["k_kv_attn_few<128, 2, false>"]),
    (256, 1, 2, 64, [1, 3], [200, 90], 50, None, ["k_kv_attn_few<256, 1, false>"]),
    (64, 1, 2, 16, [1, 1], [3000, 1700], 1301, None, ["k_kv_attn_few<64, 1, true>"]),
    (128, 1, 8, 64, [4, 4], [3000, 1700], 1303, None, ["k_kv_attn_few<128, 2, true>"]),
    (256, 1, 2, 128, [1, 1], [3000, 1700], 1301, None, ["k_kv_attn_few<256, 1, true>"]),
    (64, 1, 1, 16, [140, 1], [200, 90], 37, None, ["k_kv_attn_many<64>"]),
    (128, 2, 1, 16, [150, 130], [200, 700], 100, None, ["k_kv_attn_many<128>"]),
    (256, 1, 2, 64, [70, 1], [200, 90], 21, False, ["k_kv_attn_many<256>"]),
    (64, 1, 1, 16, [140, 1], [3000, 90], 1301, None, ["k_kv_attn_many<64>", "k_kv_attn_join"]),
    (128, 1, 1, 32, [140, 1], [3000, 90], 1301, None, ["k_kv_attn_many<128>", "k_kv_attn_join"]),
    (256, 1, 1, 64, [140, 1], [3000, 90], 1301, None, ["k_kv_attn_many<256>", "k_kv_attn_join"]),
]


@pytest.mark.parametrize("D,H,G,page,q,kv,window,workspace,kernels", WINDOWS)
def test_tokens_before_every_window_need_no_bytes(D, H, G, page, q, kv, window, workspace, kernels):
    """A prompt whose older tokens were never written (slot -1): their bytes, also those beside the
    first visible token, are all ones, whose scales stand for NaN."""
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, page, q, kv, seed=D + window)
    first = [max(0, L - n - window + 1) for n, L in zip(q, kv)]
    assert any(n % 16 for n in first), "no token beside the first visible one"
    for b, n in enumerate(first):
        fill_tokens(c, b, range(n), 255, 255)
    plan = plan_of(mx, c, window, workspace=workspace)
    assert all(k in plan for k in kernels), plan
    c.check(mx, window=window, workspace=workspace, what=plan)
