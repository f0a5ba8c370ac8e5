"""What must not reach a result of mx_kv_attention: bytes of tokens that no row sees, in every
kernel the call can take. Exact values and bounds are the float64 oracle's."""
import numpy as np
import pytest

from oracle import mx_kv_oracle as KV

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_kv import Case, _close

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


# D, H, G, page, q, kv, what the plan names: lengths that end inside pages and token tiles
ENDS = [
    (64, 2, 3, 64, [1, 4], [201, 90], ["k_kv_attn_few<64, 1, false>"]),
    (64, 1, 8, 64, [4, 4], [201, 90], ["k_kv_attn_few<64, 2, false>"]),
    (128, 2, 3, 64, [1, 4], [201, 90], ["k_kv_attn_few<128, 1, false>"]),
    (128, 1, 8, 64, [4, 4], [3001, 1700], ["k_kv_attn_few<128, 2, true>"]),
    (256, 1, 2, 64, [1, 3], [201, 90], ["k_kv_attn_few<256, 1, false>"]),
    (256, 1, 2, 64, [1, 1], [3001, 1700], ["k_kv_attn_few<256, 1, true>"]),
    (64, 1, 1, 64, [140, 1], [3001, 90], ["k_kv_attn_many<64>", "k_kv_attn_join"]),
    (128, 1, 1, 64, [140, 150], [201, 150], ["k_kv_attn_many<128>"]),
    (256, 1, 1, 64, [140, 1], [201, 90], ["k_kv_attn_many<256>"]),
]


@pytest.mark.parametrize("D,H,G,page,q,kv,kernels", ENDS)
def test_bytes_past_the_ends_change_no_bit(D, H, G, page, q, kv, kernels):
    """Whatever codes and scales stand behind a request's last token in its last page, and in pages
    that no table names, the result is the same bit for bit."""
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, page, q, kv, seed=D + sum(q))
    plan = plan_of(mx, c)
    assert all(k in plan for k in kernels), plan
    first = c.check(mx, what=plan)
    rng = np.random.default_rng(1)
    used = {int(p) for row, L in zip(c.table, kv) for p in row[:-(-L // page)]}
    for scales in (lambda *n: rng.integers(0, 256, n), lambda *n: np.full(n, 255), lambda *n: np.full(n, 254), lambda *n: np.zeros(n)):
        for b, L in enumerate(kv):
            fill_tokens(c, b, range(L, -(-L // page) * page), lambda *n: rng.integers(0, 256, n), scales)
        for p in set(range(c.pages)) - used:
            c.cache[p] = rng.integers(0, 256, c.cache[p].shape)
        assert np.array_equal(first, c.check(mx, what=plan))


@pytest.mark.parametrize("D,q,kv", [(64, [1, 3], [90, 201]), (128, [1, 3], [90, 201]), (256, [1, 3], [90, 201]),
                                    (128, [1, 1], [3001, 90]), (64, [140, 3], [201, 90]), (128, [140, 3], [1600, 90]),
                                    (256, [140, 3], [201, 90])])
@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80])
def test_queries_that_are_not_finite_stay_in_their_row(D, q, kv, value):
    """NaN and infinities in one head of one row of each request: every other row and head is right."""
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, 2, 2, 16, q, kv, seed=D, extra_rows=3)
    exact, bound = c.exact()
    n = int(c.cu[-1])
    fine = np.ones(exact.shape[:2], dtype=bool)
    fine[n:] = False
    for b in range(len(q)):
        row, head = int(c.cu[b]) + q[b] // 2, 1 + b
        c.q[row, head, 5 + 31 * b] = value
        fine[row, head] = False
    c.q[n:] = value  # rows of no request
    import torch
    out = torch.full((c.T, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_kv_attention(dev_bf16(c.q), *c.args(), out=out, max_q=max(q), max_kv=max(kv))
    _close(host_bits(out)[fine], exact[fine], bound[fine], plan_of(mx, c))
    assert bool((out[n:] == 7).all())
