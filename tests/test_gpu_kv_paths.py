"""Every kernel that mx_kv_attention can launch, at lengths where a token lost or taken twice shows:
at a seam between shares, between waves, at a refetch of pages, between splits.

Two kinds of inputs make single tokens visible among many thousands.
  - Equal weights: all keys are 0, so that every score is 0 and every weight exactly 1, and the sums of
    the values (whole numbers) and of the weights are exact in FP32. A unit of 32 tokens has its
    values in one element of the head, at most 64 units share it, and the result is off by the last
    rounding alone: 2^-8 for bf16, and 2^-21 for the division and the product before it.
  - Needles: a row's query is aligned with the keys of some tokens, the others' keys are small, and
    those tokens share about two thirds of the weight. They lie on both sides of every border of the
    shares. The bound is the oracle's, of which a needle's contribution is several times as much."""
import re

import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_kv import Case, _close, dev
from test_gpu_kv_masks import plan_of

pytestmark = pytest.mark.gpu

UNIT = 32  # tokens of a step, and of a share's unit
START = 8  # units that a segment's start and end count for

# name: D, H, G, page, q, kv, options, what the plan names
PATHS = {
    "few 64": (64, 2, 3, 16, [1, 3], [1200, 90], {}, ["k_kv_attn_few<64, 1, false>"]),
    "few 64 tall": (64, 1, 8, 16, [4, 4], [1200, 90], {}, ["k_kv_attn_few<64, 2, false>"]),
    "few 128": (128, 2, 3, 16, [1, 3], [1200, 90], {}, ["k_kv_attn_few<128, 1, false>"]),
    "few 128 tall": (128, 1, 8, 16, [4, 4], [1200, 90], {}, ["k_kv_attn_few<128, 2, false>"]),
    "few 256": (256, 1, 3, 16, [1, 3], [1200, 90], {}, ["k_kv_attn_few<256, 1, false>"]),
    "few 128 uncut": (128, 1, 16, 128, [1, 1], [40003, 90], {"workspace": False}, ["k_kv_attn_few<128, 1, false>"]),
    "few 256 uncut": (256, 1, 16, 64, [1], [9001], {"workspace": False}, ["k_kv_attn_few<256, 1, false>"]),
    # many parts a segment
    "long 64": (64, 1, 2, 128, [1, 1], [131072, 70], {}, ["k_kv_attn_few<64, 1, true> workers=512"]),
    "long 128": (128, 1, 16, 128, [1, 1], [131071, 70], {}, ["k_kv_attn_few<128, 1, true> workers=512"]),
    "shares 64": (64, 1, 16, 64, [1, 1], [40003, 70], {}, ["k_kv_attn_few<64, 1, true> workers=128"]),
    "shares 64 tall": (64, 1, 16, 64, [2, 1], [40003, 333], {}, ["k_kv_attn_few<64, 2, true> workers=128"]),
    "shares 128": (128, 1, 16, 64, [1, 1], [40003, 70], {}, ["k_kv_attn_few<128, 1, true> workers=128"]),
    "shares 128 tall": (128, 1, 8, 64, [4, 1], [40003, 333], {}, ["k_kv_attn_few<128, 2, true> workers=128"]),
    "shares 256": (256, 1, 16, 64, [1, 1], [40003, 70], {}, ["k_kv_attn_few<256, 1, true> workers=128"]),
    # few parts a segment, several segments a share
    "seams 64": (64, 8, 2, 16, [1] * 5, [3000, 1, 0, 2611, 1777], {}, ["k_kv_attn_few<64, 1, true> workers=256"]),
    "seams 128": (128, 8, 2, 16, [2] * 5, [3000, 1, 0, 2611, 1777], {}, ["k_kv_attn_few<128, 1, true> workers=256"]),
    "seams 128 tall": (128, 8, 8, 16, [4] * 4, [3000, 1, 2611, 1777], {}, ["k_kv_attn_few<128, 2, true> workers=256"]),
    "seams 256": (256, 8, 2, 16, [2] * 4, [3000, 1, 2611, 1777], {}, ["k_kv_attn_few<256, 1, true> workers=256"]),
    # many rows, one workgroup's walk and split ones
    "many 64": (64, 2, 1, 64, [150, 3], [5003, 700], {"workspace": False}, ["k_kv_attn_many<64> C=1073741824 S=1"]),
    "many 128": (128, 1, 2, 64, [150, 3], [5003, 700], {"workspace": False}, ["k_kv_attn_many<128> C=1073741824 S=1"]),
    "many 256": (256, 1, 2, 64, [90, 3], [5003, 700], {"workspace": False}, ["k_kv_attn_many<256> C=1073741824 S=1"]),
    "splits 64": (64, 2, 1, 64, [150, 3], [9003, 700], {}, ["k_kv_attn_many<64> C=576 S=16 + k_kv_attn_join"]),
    "splits 128": (128, 1, 2, 64, [150, 3], [9003, 700], {}, ["k_kv_attn_many<128> C=576 S=16 + k_kv_attn_join"]),
    "splits 256": (256, 1, 2, 64, [90, 3], [9003, 700], {}, ["k_kv_attn_many<256> C=576 S=16 + k_kv_attn_join"]),
}


def path(mx, name):
    D, H, G, page, q, kv, options, kernels = PATHS[name]
    plan = mx.mx_kv_attention_plan(len(q), sum(q), H * G, H, D, max(q), max(kv),
                                   workspace_bytes=0 if options.get("workspace") is False else None)
    assert all(k in plan for k in kernels), plan
    return PATHS[name][:6], options, plan


class Deep:
    """Requests' keys and values as payload and scales [H, tokens, ..] each, in a paged cache."""

    def __init__(self, D, H, G, page, q, kv, seed=0):
        self.D, self.H, self.G, self.page, self.q_lens, self.kv_lens = D, H, G, page, q, kv
        self.cu = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.rng = np.random.default_rng(seed)

    def put(self, k, v):
        """k, v: for each request float64 [H, L, D] that MXFP4 holds; scales are the quantizer's."""
        page, D = self.page, self.D
        each = [-(-L // page) for L in self.kv_lens]
        pages = sum(each) + 1
        ids = self.rng.permutation(pages)
        table = np.full((len(each), max(each) + 1), -1, dtype=np.int32)
        packed = []
        for x in (k, v):
            rows = np.zeros((pages, self.H, page, D), dtype=np.float32)
            at = 0
            for b, (L, n) in enumerate(zip(self.kv_lens, each)):
                table[b, :n] = ids[at:at + n]
                whole = np.zeros((self.H, n * page, D), dtype=np.float32)
                whole[:, :L] = x[b]
                rows[ids[at:at + n]] = whole.reshape(self.H, n, page, D).transpose(1, 0, 2, 3)
                at += n
            codes, scales = O.quantize_mx(W.f32_to_bf16_bits(rows.reshape(-1, D)))
            packed += [codes.reshape(pages, self.H, page, -1), scales.reshape(pages, self.H, page, -1)]
        self.table, self.cache = table, KV.pack(*packed, page)

    def run(self, mx, q_bits, **kw):
        out = mx.mx_kv_attention(dev_bf16(q_bits), dev(self.cache), dev(self.table), dev(self.cu), dev(np.array(self.kv_lens, np.int32)),
                                 self.H, self.page, max_q=max(self.q_lens), max_kv=max(self.kv_lens), **kw)
        return host_bits(out)


@pytest.mark.parametrize("name", PATHS)
@pytest.mark.parametrize("causal", [True, False])
def test_equal_weights_lose_no_token(name, causal):
    torch_or_skip()
    mx = lib_or_fail()
    (D, H, G, page, q, kv), options, plan = path(mx, name)
    c = Deep(D, H, G, page, q, kv, seed=len(name))
    values = []
    for L in kv:
        j = np.arange(L)
        v = np.zeros((H, L, D))
        for h in range(H):
            v[h, j, (j // UNIT + 7 * h) % D] = 1 + j % 4
        values.append(v)
    c.put([np.zeros((H, L, D)) for L in kv], values)
    bits = c.run(mx, W.normal_bf16((c.T, H * G, D), seed=3), causal=causal, **options)
    want = np.zeros((c.T, H, D))
    for b, (n, L) in enumerate(zip(q, kv)):
        for i in range(n):
            end = max(0, L - n + i + 1) if causal else L
            if end:
                want[c.cu[b] + i] = values[b][:, :end].sum(axis=1) / end
    want = np.repeat(want, G, axis=1)
    _close(bits, want, (2.0 ** -8 + 2.0 ** -21) * want, plan)


def borders(plan, kv, H, G, q, h):
    """The tokens of request 0's head h, first row tile, where a share, a split or a window of page
    entries begins, if the shares lie as the kernel's rule says: request after request, head fastest."""
    at = set(range(512, kv[0], 512))
    few = re.search(r"few<\d+, (\d), true> workers=(\d+)", plan)
    if few:
        R, n = 16 * int(few.group(1)), int(few.group(2))
        units = [-(-L // UNIT) + START for L in kv]
        total = sum(H * -(-m * G // R) * u for m, u in zip(q, units))
        for i in range(1, n):
            at.add(UNIT * (i * total // n - h * units[0] - START))
    split = re.search(r"many<\d+> C=(\d+)", plan)
    if split:
        at.update(range(int(split.group(1)), kv[0], int(split.group(1))))
    return sorted(x for x in at if 0 < x < kv[0] - max(q))


@pytest.mark.parametrize("name", [n for n in PATHS if not n.startswith("long")])
def test_needles_at_every_border(name):
    """Request 0, all of its heads: both sides of every border are needles of one of its rows."""
    torch_or_skip()
    mx = lib_or_fail()
    (D, H, G, page, q, kv), options, plan = path(mx, name)
    c = Deep(D, H, G, page, q, kv, seed=len(name) + 1)
    rows, L, scale = q[0] * G, kv[0], D ** -0.5
    spots = []  # of each head
    for h in range(H):
        ends = {x for b in borders(plan, kv, H, G, q, h) for x in (b - 1, b)}
        spots.append(np.array(sorted(ends | {0, 15, 16, 31, 32, L - q[0]})))
    k, v = [], []
    for b, n in enumerate(kv):
        for x, std in ((k, 0.25), (v, 1.0)):
            codes, scales = O.quantize_mx(W.normal_bf16((H * n, D), seed=10 * b + int(std), std=std))
            x.append(O.dequantize_mx(codes, scales).reshape(H, n, D))
    x = O.bf16_to_f64(W.normal_bf16((c.T, H * G, D), seed=5))
    for h in range(H):
        for r in range(rows):
            mine = spots[h][r::rows]
            sign = c.rng.choice([-1.0, 1.0], D)
            k[0][h, mine] = sign
            # e^score each, against about L others of e^0: the needles have 2/3 of the weight
            x[r // G, h * G + r % G] = sign * np.log(2.0 * L / max(len(mine), 1)) / (D * scale)
    q_bits = W.f32_to_bf16_bits(x.astype(np.float32))
    x = O.bf16_to_f64(q_bits)
    c.put(k, v)
    out = O.bf16_to_f64(c.run(mx, q_bits, **options))
    for b, (n, m) in enumerate(zip(q, kv)):
        seen = np.arange(m)[None] <= (m - n + np.arange(n))[:, None]
        at = slice(c.cu[b], c.cu[b + 1])
        for hq in range(H * G):
            h = hq // G
            if m == 0:
                assert not out[at, hq].any()
                continue
            exact, bound = KV.attend(x[at, hq], k[b][h], v[b][h], seen, scale)
            if b == 0:  # the test's own: each needle, were it lost, would leave the bound
                s = np.exp(scale * (x[at, hq] @ k[0][h].T)) * seen
                for i in range(n):
                    mine = spots[h][i * G + hq % G::rows]
                    moved = (s[i, mine] / s[i].sum())[:, None] * np.abs(v[0][h, mine] - exact[i])
                    assert (moved > 2 * bound[i]).any(axis=1).all(), "a needle too small to be seen"
            bad = ~(np.abs(out[at, hq] - exact) <= bound)
            assert not bad.any(), f"{plan}: request {b} head {hq}, row and element {np.argwhere(bad)[0]}"


# ------------------------------------------------------------------------------- many rows

MANY = [(64, None), (64, False), (128, None), (128, False), (256, None), (256, False)]


def many_rows(mx, D, workspace, seed):
    """A case whose first request and last are the many-rows kernel's, split where it has a workspace."""
    c = Case(D, 2, 2, 16, [140, 2, 70], [1500, 90, 300], seed=seed, extra_rows=2)
    plan = plan_of(mx, c, workspace=workspace)
    assert f"k_kv_attn_many<{D}>" in plan and ("k_kv_attn_join" in plan) == (workspace is None), plan
    return c


@pytest.mark.parametrize("D,workspace", MANY)
def test_many_rows_bad_pages_hide_their_tokens(D, workspace):
    torch_or_skip()
    mx = lib_or_fail()
    c = many_rows(mx, D, workspace, 31)
    c.table[0, 0], c.table[0, 37], c.table[2, 2] = c.pages, -1, 2 ** 31 - 1
    c.table[0, 93], c.table[2, 18] = -(2 ** 31), c.pages + 7   # the last pages, ragged
    c.table[0, 40:80] = -1                                     # a whole split and more
    c.check(mx, what="bad pages", workspace=workspace)
    c.check(mx, causal=False, what="bad pages, all", workspace=workspace)
    c.table[:] = -1
    assert not c.check(mx, what="no page at all", workspace=workspace)[:212].any()


@pytest.mark.parametrize("D,workspace", MANY)
def test_many_rows_of_shared_pages(D, workspace):
    torch_or_skip()
    mx = lib_or_fail()
    c = many_rows(mx, D, workspace, 32)
    c.table[2, :9] = c.table[0, :9]
    c.table[0, 50] = c.table[0, 11]
    c.check(mx, what="shared", workspace=workspace)


@pytest.mark.parametrize("D,workspace", MANY)
def test_many_rows_strided_rows_and_output(D, workspace):
    torch = torch_or_skip()
    mx = lib_or_fail()
    c = many_rows(mx, D, workspace, 33)
    n = int(c.cu[-1])
    wide = torch.full((c.T, 7, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = dev_bf16(c.q)
    exact, bound = c.exact()
    home = torch.full((c.T, 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mx_kv_attention(wide[:, 2:6], *c.args(), out=home[:, 1:5], max_q=140, max_kv=1500, workspace=workspace)
    _close(host_bits(home[:n, 1:5]), exact[:n], bound[:n], "strided")
    assert bool((home[:, 0] == 7).all()) and bool((home[:, 5] == 7).all()) and bool((home[n:] == 7).all())


@pytest.mark.parametrize("D,workspace", MANY)
def test_many_rows_garbage_lengths_stay_in_bounds(D, workspace):
    torch = torch_or_skip()
    mx = lib_or_fail()
    c = many_rows(mx, D, workspace, 34)
    cache, table, cu, kv, H, page = c.args()
    for cu_bad, kv_bad in (([0, 140, 142, 9999], [1500, 90, 300]), ([-5, 140, 142, 212], [1500, 2 ** 31 - 1, -7]),
                           ([0, 200, 3, 214], [1500] * 3), ([2 ** 31 - 1] * 4, [1] * 3), ([-2 ** 31] * 4, [1] * 3)):
        guard = torch.full((c.T + 2, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.mx_kv_attention(dev_bf16(c.q), cache, table, dev(np.array(cu_bad, np.int32)), dev(np.array(kv_bad, np.int32)), H, page,
                           out=guard[1:c.T + 1], max_q=140, max_kv=1500, workspace=workspace)
        torch.cuda.synchronize()
        assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_beyond_the_lanes_of_a_wave(D):
    """More than 64 requests of many rows, ragged, beside short and empty ones: their order is no longer
    sorted by length."""
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(D)
    q = [int(x) for x in rng.integers(0, 3, 70) * rng.integers(0, 100, 70)]
    q[9] = 300
    kv = [n + int(x) for n, x in zip(q, rng.integers(0, 90, 70))]
    c = Case(D, 1, 1, 16, q, kv, seed=D + 35, extra_rows=1)
    assert "k_kv_attn_many" in plan_of(mx, c)
    c.check(mx, what="70 requests")
