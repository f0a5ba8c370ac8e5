"""GPU parity of routing, its tables, the cache's append and the verification of drafts against the
float64 oracle (oracle/mx_step_oracle.py).

Choices, tables, cache bytes and tokens are compared exactly. Routing weights are formed in FP64 and
rounded once: half a step of FP32, 2^-24 of the value (and 2^-40 for the FP64 sums of at most 1024
terms). Rotated queries are held to the bound that the oracle derives from the arithmetic. Nothing here
comes from a measured error."""
import math

import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O
from oracle import mx_step_oracle as S

from gpu_util import check_gemm, dev_bf16, host_bits, lib_or_fail, torch_or_skip

pytestmark = pytest.mark.gpu


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------------------- routing

def _check_route(mx, logits, topk, f32, bias=None, lead=0, pad=0, rows=None, sigmoid=False, what="", **kw):
    """logits: float32 values (bf16 ones unless f32); lead: elements before the first row, pad: between rows."""
    import torch
    T, E = logits.shape
    want, weights = S.route(logits, topk, bias=bias, sigmoid=sigmoid, rows=rows, largest=S.FLT_MAX if f32 else S.BF16_MAX, **kw)
    home = np.full((lead + T * (E + pad),), np.nan, np.float32)
    view = home[lead:].reshape(T, E + pad)
    view[:, :E] = logits
    d = dev(home) if f32 else dev_bf16(W.f32_to_bf16_bits(np.nan_to_num(home, nan=9.0, posinf=np.inf, neginf=-np.inf)))
    if not f32:
        d[lead:].view(T, E + pad)[:, :E][dev(np.isnan(logits))] = math.nan
    d = d[lead:].view(T, E + pad)[:, :E]
    ids = torch.full((T + 2, topk), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, topk), 77.0, dtype=torch.float32, device="cuda")
    mx.mx_moe_route(d, topk, bias=None if bias is None else dev(np.asarray(bias, np.float32)),
                    score=mx.MX_SCORE_SIGMOID if sigmoid else mx.MX_SCORE_SOFTMAX,
                    num_rows=None if rows is None else dev(np.array([rows], np.int32)), ids=ids[:T], weights=w[:T], **kw)
    got, gw = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.all(got[T:] == 77) and np.all(gw[T:] == 77)
    bad = np.argwhere(got[:T] != want)
    assert bad.size == 0, (what, bad[0], got[bad[0][0]], want[bad[0][0]])
    assert np.all(np.abs(gw[:T] - weights) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(weights) + 2.0 ** -149), what


def _logits(T, E, seed, f32, std=2.0):
    x = W.normal_bf16((T, E), seed, std)
    x = W.bf16_bits_to_f32(x)
    return x + np.float32(2.0 ** -12) * W.bf16_bits_to_f32(W.normal_bf16((T, E), seed + 1)) if f32 else x


@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (7, 8, 8), (3, 1, 1), (5, 60, 4), (130, 64, 6), (33, 128, 8), (64, 160, 6), (257, 256, 8),
                                      (50, 384, 64), (16, 896, 16), (70, 896, 16), (9, 1000, 33), (4, 1024, 64), (11, 1023, 7), (300, 17, 3)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route(T, E, topk, f32, sigmoid):
    torch_or_skip()
    mx = lib_or_fail()
    x = _logits(T, E, T + E, f32)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.2).astype(np.float32)
    _check_route(mx, x, topk, f32, sigmoid=sigmoid)
    _check_route(mx, x, topk, f32, sigmoid=sigmoid, bias=bias, renormalize=False, scale=2.5, lead=1, pad=3, rows=T - T // 3)
    _check_route(mx, x, topk, f32, sigmoid=sigmoid, renormalize=False, scale=-0.75, lead=8, pad=8)
    _check_route(mx, x, topk, f32, sigmoid=sigmoid, bias=bias)


@pytest.mark.parametrize("E,groups,keep,topk", [(8, 4, 2, 3), (64, 8, 3, 8), (160, 8, 3, 6), (256, 8, 4, 8), (256, 32, 5, 16), (512, 16, 1, 20),
                                                (1000, 5, 2, 9), (960, 3, 2, 16), (896, 56, 11, 16), (64, 64, 9, 9), (1024, 2, 1, 64), (60, 12, 12, 4),
                                                (1008, 63, 7, 8), (6, 1, 1, 2)])
@pytest.mark.parametrize("f32", [False, True])
def test_route_in_groups(E, groups, keep, topk, f32):
    torch_or_skip()
    mx = lib_or_fail()
    x = _logits(41, E, E + groups, f32)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.1).astype(np.float32)
    for sigmoid in (False, True):
        for top in (1, 2):
            for b in (None, bias):
                _check_route(mx, x, topk, f32, sigmoid=sigmoid, groups=groups, topk_groups=keep, group_top=top, bias=b, renormalize=top == 2,
                             lead=8 * (E % 3), what=(sigmoid, top, b is None))


@pytest.mark.parametrize("E,groups,keep,topk", [(16, 1, 1, 5), (64, 8, 4, 8), (256, 8, 3, 8), (896, 1, 1, 16), (1000, 50, 3, 12)])
def test_route_ties_go_to_the_lower(E, groups, keep, topk):
    """Logits of few values, so that most comparisons are ties, among groups too."""
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(E)
    x = rng.integers(-1, 2, (60, E)).astype(np.float32)
    x[0] = 0
    x[1] = -0.0
    x[2] = np.where(rng.random(E) < 0.5, 0.0, -0.0)
    x[3] = -3
    bias = rng.integers(-1, 2, E).astype(np.float32) * 0.25
    for sigmoid in (False, True):
        for b in (None, bias, 0 * bias, -2 + 0 * bias):
            for top in (1, 2):
                for f32 in (False, True):
                    _check_route(mx, x, topk, f32, sigmoid=sigmoid, groups=groups, topk_groups=keep, group_top=top, bias=b, what=(sigmoid, top))


@pytest.mark.parametrize("E,groups,keep,topk", [(8, 1, 1, 4), (64, 8, 4, 8), (256, 1, 1, 8), (896, 7, 2, 16), (160, 8, 3, 30)])
@pytest.mark.parametrize("f32", [False, True])
def test_route_of_masked_infinite_and_nan_logits(E, groups, keep, topk, f32):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(E + topk)
    x = _logits(40, E, E, f32)
    x[rng.random(x.shape) < 0.2] = -np.inf
    x[rng.random(x.shape) < 0.05] = np.nan
    x[3:8, rng.random(E) < 0.9] = -np.inf
    x[8] = -np.inf
    x[9] = np.nan
    x[10, :] = -np.inf
    x[10, E // 2] = 1
    x[11, rng.random(E) < 0.3] = np.inf
    x[12, E - 1] = np.inf
    x[13] = W.bf16_bits_to_f32(np.array([0xFF7F], np.uint16))[0]   # the type's lowest value
    x[14, ::2] = W.bf16_bits_to_f32(np.array([0xFF7F], np.uint16))[0]
    x[15] = W.bf16_bits_to_f32(np.array([0x7F7F], np.uint16))[0]
    x[16] = x[16] * 32                                             # exact in bf16: scores that vanish or saturate
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    off = bias.copy()
    off[rng.random(E) < 0.3] = -np.inf
    off[0] = np.nan
    for sigmoid in (False, True):
        for b in (None, bias, off):
            for renormalize in (False, True):
                _check_route(mx, x, topk, f32, sigmoid=sigmoid, groups=groups, topk_groups=keep, bias=b, renormalize=renormalize,
                             what=(sigmoid, b is None, renormalize))
    off[:] = -np.inf
    _check_route(mx, x, topk, f32, bias=off, groups=groups, topk_groups=keep)
    off[E // 2], off[0] = np.inf, 1e30
    _check_route(mx, x, topk, f32, bias=off, groups=groups, topk_groups=keep)


def test_route_rows_of_padding_and_of_nothing():
    torch = torch_or_skip()
    mx = lib_or_fail()
    x = _logits(37, 64, 1, False)
    for rows in (-4, 0, 1, 36, 37, 1000):
        _check_route(mx, x, 6, False, rows=rows, bias=np.zeros(64))
    ids, w = mx.mx_moe_route(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), 4)
    assert ids.shape == w.shape == (0, 4)
    # one row for all tokens
    one = dev_bf16(W.normal_bf16((1, 64), 3)).expand(9, 64)
    ids, w = mx.mx_moe_route(one, 4)
    assert bool((ids == ids[:1]).all()) and bool((w == w[:1]).all())


# ------------------------------------------------------------------------------- sort

def _check_sort(mx, ids, E, first=0):
    import torch
    T, topk = ids.shape
    want = S.sort(ids, E, first)
    out = [torch.full((n + 3,), 77, dtype=torch.int32, device="cuda") for n in (E + 1, T * topk, T * topk)]
    nbytes = mx.mx_moe_sort_workspace_bytes(T, topk, E)
    ws = torch.full((nbytes + 64,), 171, dtype=torch.uint8, device="cuda")
    mx.mx_moe_sort(dev(ids.astype(np.int32)), E, first_expert=first, expert_offsets=out[0][:E + 1], row_token=out[1][:T * topk],
                   token_rows=out[2][:T * topk].view(T, topk), workspace=ws[:nbytes] if nbytes else None)
    got = [x.cpu().numpy() for x in out]
    for name, g, w in zip(("expert_offsets", "row_token", "token_rows"), got, want):
        assert np.array_equal(g[:w.size], w.reshape(-1)), name
        assert np.all(g[w.size:] == 77), name
    assert bool((ws[nbytes:] == 171).all())
    for g, w in zip(mx.mx_moe_sort(dev(ids.astype(np.int32)), E, first_expert=first), want):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("T,topk,E", [(1, 1, 1), (1, 16, 896), (16, 16, 896), (3, 2, 8), (256, 16, 896), (1000, 8, 64), (63, 1, 1024), (65, 3, 1023),
                                      (2048, 8, 256), (2049, 8, 256), (4096, 16, 896), (4000, 4, 8), (20000, 1, 60), (70001, 6, 160),
                                      (5, 1024, 1024), (600000, 8, 128)])
@pytest.mark.parametrize("kind", ["even", "one", "skewed"])
def test_sort(T, topk, E, kind):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(T + E)
    if kind == "even":
        ids = rng.integers(0, E, (T, topk))
    elif kind == "one":
        ids = np.full((T, topk), E - 1)
    else:
        ids = np.minimum((rng.random((T, topk)) ** 4 * E).astype(np.int64), E - 1)
        ids[rng.random(ids.shape) < 0.1] = -1
    _check_sort(mx, ids, E)
    _check_sort(mx, ids, max(1, E // 3), first=E // 4)


def test_sort_of_ids_out_of_range_and_of_nothing():
    torch = torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(1)
    for T in (50, 9000):
        ids = rng.integers(-3, 12, (T, 4))
        ids[0], ids[1] = [2 ** 31 - 1, -2 ** 31, 8, 7], [-1, -2, 0, 100000]
        _check_sort(mx, ids, 8)
        _check_sort(mx, ids, 4, first=(1 << 30) - 1)
        _check_sort(mx, np.full((T, 4), -1), 8)
    for E in (1, 1024):
        off, tok, rows = mx.mx_moe_sort(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), E)
        assert off.tolist() == [0] * (E + 1) and tok.numel() == 0 and rows.shape == (0, 4)


# ------------------------------------------------------------------------------- append

def _check_append(mx, T, Hq, H, D, page, seed=0, pairs=False, rot=None, norms=True, order="random", layout="fused", rope_scale=1.0, eps=1e-6,
                  positions=None, std=1.0, in_place=False, with_kv=True, base=10000.0):
    import torch
    rng = np.random.default_rng(seed + T + D)
    rot = D if rot is None else rot
    bits = W.normal_bf16((T, Hq + 2 * H, D), seed, std)
    if T > 2 and H:
        bits[1, Hq:, :32] = 0                                # blocks of zeros
        bits[2, Hq:, 32:64] = 0x8000
    pages = -(-T // page) + 2
    slots = (rng.permutation(pages * page)[:T] if order == "random" else np.arange(T) + page // 3).astype(np.int64)
    pos = rng.integers(0, 100000, T) if positions is None else np.asarray(positions)
    pos = pos.astype(np.int32)
    if T > 6:
        slots[3], slots[5] = -1, pages * page                # no slot: the queries are still done
        pos[4], pos[6] = -1, -2 ** 31                        # padding
    freq = None if rot == 0 else (base ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)
    qw, kw = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    if norms is False:
        qw = kw = None
    elif norms == "q":
        kw = None
    wide = dev_bf16(bits)
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + H], wide[:, Hq + H:]
    if layout == "dense":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out = torch.full((T + 1, Hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out_bits = host_bits(out)[:T, :Hq].copy()
    if in_place:
        out, out_bits = q, bits[:, :Hq].copy()
    start = rng.integers(0, 256, (pages, max(H, 1), KV.block_bytes(page, D)), dtype=np.uint8)
    cache = dev(start)
    call = dict(inv_freq=None if freq is None else dev(freq), rope=mx.MX_ROPE_PAIRS if pairs else mx.MX_ROPE_HALVES, rope_scale=rope_scale, eps=eps,
                q_weight=None if qw is None else dev(qw), k_weight=None if kw is None else dev(kw))
    kv = (k, v, dev(pos), dev(slots), cache) if with_kv else (None, None, dev(pos), None, None)
    got = mx.mx_kv_append(q if Hq else None, *kv, page, q_out=out[:T, :Hq] if Hq else None, **call)
    live = pos >= 0
    if Hq:
        y, size = S.norm_rotate(O.bf16_to_f64(bits[:, :Hq]), pos, qw, eps, freq, pairs, rope_scale)
        g = host_bits(got)
        err, bound = np.abs(O.bf16_to_f64(g) - y), S.query_bound(y, size)
        bad = np.argwhere((err > bound)[live])
        assert bad.size == 0, (bad[0], err[live][tuple(bad[0])], bound[live][tuple(bad[0])])
        assert np.array_equal(g[~live], out_bits[~live])
        if not in_place:
            assert bool((out[T:] == 7).all()) and bool((out[:, Hq:] == 7).all())
        elif H:
            assert np.array_equal(host_bits(wide)[:, Hq:], bits[:, Hq:])
    else:
        assert got is None
    if with_kv:
        want = start.copy()
        S.append(want, O.bf16_to_f64(bits[:, Hq:Hq + H]), bits[:, Hq + H:], pos, slots, page, kw, eps, freq, pairs, rope_scale)
        assert np.array_equal(cache.cpu().numpy(), want)
    else:
        assert np.array_equal(cache.cpu().numpy(), start)


@pytest.mark.parametrize("T,Hq,H,D,page", [(1, 4, 1, 64, 16), (1, 32, 8, 128, 16), (5, 3, 3, 64, 32), (37, 10, 5, 128, 64), (101, 32, 8, 128, 16),
                                           (70, 7, 7, 64, 128), (19, 4, 2, 256, 16), (131, 5, 1, 256, 1024), (600, 8, 2, 128, 32), (2500, 2, 1, 64, 16)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("order", ["random", "run"])
def test_append(T, Hq, H, D, page, pairs, order):
    torch_or_skip()
    mx = lib_or_fail()
    _check_append(mx, T, Hq, H, D, page, pairs=pairs, order=order)
    _check_append(mx, T, Hq, H, D, page, seed=1, pairs=pairs, order=order, norms=False, rot=D // 2, layout="dense")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_rotations_and_norms(D, pairs):
    torch_or_skip()
    mx = lib_or_fail()
    for rot in range(0, D + 1, 16):
        _check_append(mx, 21, 3, 2, D, 16, seed=rot, pairs=pairs, rot=rot, norms=[True, False, "q"][rot // 16 % 3], rope_scale=1 + rot / 64)
    # positions so far that FP32 angles would be off by radians, and none
    far = [0, 1, 2, 3, 4, 5, 6, 2 ** 31 - 1, 2 ** 30 - 1, 2 ** 24 + 1, 131071, 10 ** 6 + 3]
    for norms in (True, False):
        _check_append(mx, 12, 3, 2, D, 16, seed=9, pairs=pairs, norms=norms, positions=far, base=500000.0)
        _check_append(mx, 12, 3, 2, D, 16, seed=9, pairs=pairs, norms=norms, positions=far, base=1.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_queries_or_keys_alone_and_in_place(D):
    torch_or_skip()
    mx = lib_or_fail()
    _check_append(mx, 45, 0, 3, D, 16)
    _check_append(mx, 45, 6, 0, D, 16, with_kv=False)
    for pairs in (False, True):
        _check_append(mx, 45, 6, 2, D, 16, in_place=True, pairs=pairs)
        _check_append(mx, 45, 5, 0, D, 16, in_place=True, with_kv=False, pairs=pairs, rot=D // 2, layout="dense")


@pytest.mark.parametrize("std,eps", [(1e18, 1e-6), (1e30, 0.0), (1e-18, 0.0), (1e-18, 1e-6), (1e-30, 1e-5)])
def test_append_norms_of_very_large_and_small_heads(std, eps):
    """Squares past FP32's range on both sides."""
    torch_or_skip()
    mx = lib_or_fail()
    _check_append(mx, 20, 3, 2, 128, 16, std=std, eps=eps)
    _check_append(mx, 20, 3, 2, 64, 16, std=std, eps=eps, norms=False)


def test_append_of_many_heads_and_of_nothing():
    torch = torch_or_skip()
    mx = lib_or_fail()
    _check_append(mx, 3, 1024, 1, 64, 16)
    _check_append(mx, 3, 1, 1024, 64, 16)
    _check_append(mx, 2, 300, 100, 128, 16)
    _check_append(mx, 2, 100, 33, 256, 16)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(mx.mx_kv_cache_bytes(1, 16, 4, 64), dtype=torch.uint8, device="cuda")
    e32, e64 = (torch.zeros(0, dtype=d, device="cuda") for d in (torch.int32, torch.int64))
    assert mx.mx_kv_append(q, q, q, e32, e64, cache, 16).shape == (0, 4, 64)
    # every row padding
    _check_append(mx, 5, 2, 2, 64, 16, positions=[-1] * 5)


def test_append_equals_the_write_of_what_needs_no_norm_and_rotation():
    """At position 0 without norms the cache gets the bytes of mx_kv_write."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    for T, H, D, page in ((300, 8, 128, 64), (77, 3, 64, 16), (50, 2, 256, 32)):
        k, v = dev_bf16(W.normal_bf16((T, H, D), 1, 3.0)), dev_bf16(W.normal_bf16((T, H, D), 2))
        slots = dev(np.random.default_rng(0).permutation(T + 9)[:T].astype(np.int64))
        pages = -(-(T + 9) // page)
        a = torch.zeros((pages, H, KV.block_bytes(page, D)), dtype=torch.uint8, device="cuda")
        b = a.clone()
        mx.mx_kv_write(k, v, slots, a, page)
        mx.mx_kv_append(None, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), slots, b, page,
                        inv_freq=torch.ones(D // 2, device="cuda"))
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------- verification

def _check_verify(mx, p, q, tokens, cu, kv, accept, sample, pads=(0, 0), what=""):
    import torch
    T, V = p.shape
    want = S.verify(p, q, tokens, cu, kv, accept, sample)

    def rows(x, pad):
        if x is None:
            return None
        home = np.full((T, V + pad), np.nan, np.float32)
        home[:, :V] = x
        return dev(home)[:, :V]

    out = [torch.full((n + 3,), 77, dtype=torch.int32, device="cuda") for n in (T, len(kv), len(kv))]
    nbytes = mx.mx_verify_drafts_workspace_bytes(len(kv), V)
    ws = torch.full((nbytes + 64,), 171, dtype=torch.uint8, device="cuda")
    args = (rows(p, pads[0]), rows(q, pads[1]), dev(np.asarray(tokens, np.int32)), dev(np.asarray(cu, np.int32)), dev(np.asarray(kv, np.int32)),
            dev(np.asarray(accept, np.float32)), dev(np.asarray(sample, np.float32)))
    mx.mx_verify_drafts(*args, out_tokens=out[0][:T], accepted=out[1][:len(kv)], new_lens=out[2][:len(kv)], workspace=ws[:nbytes])
    for name, g, w in zip(("out_tokens", "accepted", "new_lens"), out, want):
        g = g.cpu().numpy()
        assert np.array_equal(g[:w.size], w), (what, name, g[:w.size], w)
        assert np.all(g[w.size:] == 77), name
    assert bool((ws[nbytes:] == 171).all())
    for g, w in zip(mx.mx_verify_drafts(*args), want):
        assert np.array_equal(g.cpu().numpy(), w)
    return want


def _verify_inputs(rows, V, seed, pad_rows=2, std=2.0):
    rng = np.random.default_rng(seed)
    T = int(sum(rows)) + pad_rows
    soft = lambda z: (np.exp(z) / np.exp(z).sum(1, keepdims=True)).astype(np.float32)  # noqa: E731
    z = rng.standard_normal((T, V)) * std
    p, q = soft(z), soft(z + rng.standard_normal((T, V)) * 0.5)
    tokens = rng.integers(0, V, T)
    for t in range(T - 1):
        if rng.random() < 0.9:
            tokens[t + 1] = min(int(np.searchsorted(np.cumsum(q[t].astype(np.float64)), rng.random())), V - 1)
    cu = np.concatenate([[0], np.cumsum(rows)])
    return p, q, tokens, cu, rng.integers(20, 90, len(rows)) + np.array(rows), rng.random(T).astype(np.float32), rng.random(len(rows)).astype(np.float32)


@pytest.mark.parametrize("rows,V", [([1], 5), ([5], 1), ([3, 0, 1, 6], 50), ([4] * 7, 1000), ([130, 2, 66], 33), ([2, 9], 2049), ([6], 40003), ([3, 4], 65536),
                                    ([1] * 40 + [5] * 60, 3001), ([2] * 3000, 20)])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify(rows, V, sampled):
    torch_or_skip()
    mx = lib_or_fail()
    seen = set()
    for seed in range(3):
        p, q, *rest = _verify_inputs(rows, V, seed + V)
        want = _check_verify(mx, p, q if sampled else None, *rest)
        seen |= set((np.array(rows) - want[1]).tolist())
        _check_verify(mx, p, q if sampled else None, *rest, pads=(3, 3))
        _check_verify(mx, p, q if sampled else None, *rest, pads=(1, 0))
        _check_verify(mx, p, q if sampled else None, *rest, pads=(4, 8))
    if sampled and max(rows) > 1 and V > 20:  # some drafts taken, some refused
        assert len(seen) > 1


def test_verify_at_the_borders_of_its_numbers():
    torch_or_skip()
    mx = lib_or_fail()
    for V in (7, 5000):
        p, q, tokens, cu, kv, accept, sample = _verify_inputs([4, 4, 1, 3], V, V)
        for name, value in (("zero", 0.0), ("one less", 1 - 2.0 ** -24), ("one", 1.0), ("past", 3.0), ("below", -1.0), ("nan", np.nan)):
            _check_verify(mx, p, q, tokens, cu, kv, accept, np.full_like(sample, value), what=name)
            _check_verify(mx, p, q, tokens, cu, kv, np.full_like(accept, value), sample, what=name)
        same = np.full_like(accept, 0.999)
        assert _check_verify(mx, p, p, tokens, cu, kv, same, sample)[1].tolist() == [3, 3, 0, 2]   # never refused
        # equal weights and numbers that fall on their borders: the token after the border
        flat = np.full_like(p, 0.25)
        edges = (np.arange(4) / 4).astype(np.float32)
        _check_verify(mx, flat, None, tokens, cu, kv, accept, edges)
        # rows that are masked down to one token, or to none, or hold no probabilities
        one = np.zeros_like(p)
        one[:, V - 1] = 1e-30
        _check_verify(mx, one, None, tokens, cu, kv, accept, sample)
        _check_verify(mx, one, q, np.full_like(tokens, V - 1), cu, kv, accept, sample)
        _check_verify(mx, 0 * p, q, tokens, cu, kv, accept, sample)
        _check_verify(mx, np.where(p < np.median(p), np.nan, -p), q, tokens, cu, kv, accept, sample)
        odd = np.where(np.random.default_rng(V).random(p.shape) < 0.3, np.nan, p).astype(np.float32)
        _check_verify(mx, odd, q, tokens, cu, kv, accept, sample)
        _check_verify(mx, p, odd, tokens, cu, kv, accept, sample)
        # drafts out of range
        for bad in (-1, V, 2 ** 31 - 1, -2 ** 31):
            t2 = tokens.copy()
            t2[2] = t2[5] = bad
            for d in (q, None):
                _check_verify(mx, p, d, t2, cu, kv, 0 * accept, sample)
        # tables that leave the rows: clamped
        _check_verify(mx, p, q, tokens, [0, 4, 4, 9, 4000], kv, accept, sample)
        _check_verify(mx, p, q, tokens, [-5, 2, 2, 3, 6], kv, accept, sample)


def test_verify_of_nothing_and_in_place():
    torch = torch_or_skip()
    mx = lib_or_fail()
    p, q, tokens, cu, kv, accept, sample = _verify_inputs([2, 3], 100, 1)
    args = [dev(p), dev(q), dev(tokens.astype(np.int32)), dev(cu.astype(np.int32)), dev(kv.astype(np.int32)), dev(accept), dev(sample)]
    want = S.verify(p, q, tokens, cu, kv, accept, sample)
    mx.mx_verify_drafts(*args, new_lens=args[4])
    assert np.array_equal(args[4].cpu().numpy(), want[2])
    none = [args[0], args[1], args[2], args[3][:1], args[4][:0], args[5], args[6][:0]]
    out, acc, lens = mx.mx_verify_drafts(*none)
    assert out.tolist() == [-1] * len(tokens) and acc.numel() == lens.numel() == 0
    z = torch.zeros((0, 100), device="cuda")
    out, acc, lens = mx.mx_verify_drafts(z, None, args[2][:0], torch.zeros(4, dtype=torch.int32, device="cuda"), args[2][:3], args[5][:0], args[5][:3])
    assert out.numel() == 0 and acc.tolist() == [0] * 3 and torch.equal(lens, args[2][:3])


# ------------------------------------------------------------------------------- together

def test_a_layers_experts_from_logits_to_output():
    """route, sort, the grouped products and the combine, on a padded batch; against the oracle step by step."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    T, live, E, topk, K, N, K2, N2 = 45, 41, 12, 3, 256, 512, 256, 256
    a = W.normal_bf16((T, K), 1)
    w1 = [W.normal_bf16((N, K), 10 + e, 0.05) for e in range(E)]
    w2 = [W.normal_bf16((N2, K2), 50 + e, 0.05) for e in range(E)]
    p1 = torch.cat([mx.mx_prepare_weight(dev_bf16(w)) for w in w1])
    p2 = torch.cat([mx.mx_prepare_weight(dev_bf16(w)) for w in w2])
    logits = _logits(T, E, 5, False)
    bias = np.linspace(-0.1, 0.1, E).astype(np.float32)
    ids, wts = mx.mx_moe_route(dev_bf16(W.f32_to_bf16_bits(logits)), topk, bias=dev(bias), score=mx.MX_SCORE_SIGMOID, groups=4, topk_groups=2,
                               scale=2.0, num_rows=dev(np.array([live], np.int32)))
    offsets, row_token, token_rows = mx.mx_moe_sort(ids, E)
    R_max = T * topk
    x = dev_bf16(a)
    hq, hs = mx.mx_a4w4_gemm_grouped_act_quant(x, row_token, offsets, E, R_max, p1, N, rows_hint=8)
    y = torch.zeros((R_max, N2), dtype=torch.bfloat16, device="cuda")
    mx.mx_a4w4_gemm_grouped_mx(hq, hs, offsets, E, R_max, p2, N2, rows_hint=8, out=y)
    out = mx.mx_moe_combine(y, token_rows, wts)
    want_ids, want_w = S.route(logits, topk, bias=bias, sigmoid=True, groups=4, topk_groups=2, scale=2.0, rows=live)
    want_off, want_tok, want_rows = S.sort(want_ids, E)
    assert np.array_equal(ids.cpu().numpy(), want_ids) and np.array_equal(offsets.cpu().numpy(), want_off)
    assert np.array_equal(row_token.cpu().numpy(), want_tok) and np.array_equal(token_rows.cpu().numpy(), want_rows)
    R = int(want_off[-1])
    assert R == live * topk
    # the second product on the rows the first one left, and the sum over them
    h, s = hq.cpu().numpy()[:R], hs.cpu().numpy()[:R]
    exact = O.grouped_gemm_mx_ref(h, s, want_off, lambda e: w2[int(e)], rows=np.arange(R))
    check_gemm(host_bits(y)[:R], exact, what="second product")
    yb, ob = O.bf16_to_f64(host_bits(y)), O.bf16_to_f64(host_bits(out))
    for t in range(T):
        terms = [want_w[t, j] * yb[want_rows[t, j]] for j in range(topk) if want_rows[t, j] >= 0]
        total = sum(terms, np.zeros(N2))
        size = sum((np.abs(v) for v in terms), np.zeros(N2))
        assert np.all(np.abs(ob[t] - total) <= 2.0 ** -8 * np.abs(total) + (topk + 3) * 2.0 ** -24 * size * (1 + 2.0 ** -8))
    assert np.all(ob[live:] == 0)
    # the first product's rows against a call with tables made on the host
    hq2, hs2 = mx.mx_a4w4_gemm_grouped_act_quant(x, dev(want_tok), dev(want_off), E, R_max, p1, N, rows_hint=8)
    assert torch.equal(hq2[:R], hq[:R]) and torch.equal(hs2[:R], hs[:R])


class Loop:
    """A few steps of decoding with drafts over one layer's cache: tables, append, attention, verification,
    tables again with the refused drafts taken back. Everything between the steps stays on the device."""

    def __init__(self, mx, B=5, drafts=3, H=2, G=4, D=64, page=16, V=300, seed=0):
        import torch
        self.mx, self.B, self.n, self.H, self.G, self.D, self.page, self.V = mx, B, drafts + 1, H, G, D, page, V
        rng = np.random.default_rng(seed)
        self.width, self.T = 6, B * (drafts + 1) + 2
        self.pages = B * self.width
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device="cuda")
        self.stack = dev(rng.permutation(self.pages).astype(np.int32))
        self.count = dev(np.array([self.pages], np.int32))
        self.cache = torch.full((self.pages, H, KV.block_bytes(page, D)), 255, dtype=torch.uint8, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.freq = dev((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
        self.qw, self.kw = (dev((1 + 0.2 * rng.standard_normal(D)).astype(np.float32)) for _ in range(2))
        self.new = torch.zeros_like(self.lens)

    def inputs(self, step):
        p, q, tokens, _, _, accept, sample = _verify_inputs([self.n] * self.B, self.V, 100 + step, pad_rows=2)
        qkv = W.normal_bf16((self.T, self.H * (self.G + 2), self.D), 200 + step)
        return qkv, p, q, tokens.astype(np.int32), accept, sample

    def step(self, qkv, p, q, tokens, accept, sample):
        mx, Hq, H = self.mx, self.H * self.G, self.H
        self.new.copy_(self.lens + self.n)
        cu, slots, pos, _, status = mx.mx_kv_tables(self.lens, self.new, self.table, self.stack, self.count, self.page, self.T,
                                                    free_count_out=self.count)
        x = mx.mx_kv_append(qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:], pos, slots, self.cache, self.page, inv_freq=self.freq,
                            q_weight=self.qw, k_weight=self.kw)
        o = mx.mx_kv_attention(x, self.cache, self.table, cu, self.new, H, self.page, max_q=self.n, max_kv=self.width * self.page)
        out, acc, kept = mx.mx_verify_drafts(p, q, tokens, cu, self.new, accept, sample)
        *_, back = mx.mx_kv_tables(self.new, kept, self.table, self.stack, self.count, self.page, 0, free_count_out=self.count)
        self.lens.copy_(kept)
        return o, out, acc, kept, status, back


def test_steps_of_decoding_with_drafts():
    torch_or_skip()
    mx = lib_or_fail()
    L = Loop(mx)
    B, n, Hq, H, D, page = L.B, L.n, L.H * L.G, L.H, L.D, L.page
    table, stack, count = L.table.cpu().numpy(), L.stack.cpu().numpy(), L.pages
    cache, lens = L.cache.cpu().numpy(), np.zeros(B, np.int32)
    freq, qw, kw = (x.cpu().numpy() for x in (L.freq, L.qw, L.kw))
    for step in range(6):
        qkv, p, q, tokens, accept, sample = L.inputs(step)
        o, out, acc, kept, status, back = L.step(dev_bf16(qkv), *(dev(x) for x in (p, q, tokens, accept, sample)))
        new = lens + n
        cu, slots, pos, count, st, table, stack = KV.tables(lens, new, table, stack, count, page, L.T)
        assert st == int(status[0]) == int(back[0]) == 0
        S.append(cache, O.bf16_to_f64(qkv[:, Hq:Hq + H]), qkv[:, Hq + H:], pos, slots, page, kw, 1e-6, freq, False)
        assert np.array_equal(L.cache.cpu().numpy(), cache)
        y, size = S.norm_rotate(O.bf16_to_f64(qkv[:, :Hq]), pos, qw, 1e-6, freq, False)
        # attention of the exact queries: those in bf16 are off by query_bound, which moves scores by at most
        # scale * sum |bound K| and so each weight by twice that factor
        live = int(cu[-1])
        exact, bound = KV.attention(y[:live], cache, table, cu, new, page, True, 0, D ** -0.5)
        k_all, v_all = KV.read(cache, [int(table[b, i // page]) * page + i % page for b in range(B) for i in range(int(new[b]))], page, D)
        shift = D ** -0.5 * S.query_bound(y, size)[:live].sum(-1).max() * np.abs(k_all).max()
        more = np.expm1(2 * shift) * np.abs(v_all).max()
        assert np.all(np.abs(O.bf16_to_f64(host_bits(o))[:live] - exact) <= bound + more * (1 + 2.0 ** -7))
        w_out, w_acc, w_lens = S.verify(p, q, tokens, cu, new, accept, sample)
        for g, w in ((out, w_out), (acc, w_acc), (kept, w_lens)):
            assert np.array_equal(g.cpu().numpy(), w)
        _, _, _, count, st, table, stack = KV.tables(new, w_lens, table, stack, count, page, 0)
        assert st == 0 and int(L.count[0]) == count
        assert np.array_equal(L.table.cpu().numpy(), table) and np.array_equal(L.stack.cpu().numpy(), stack)
        lens = w_lens


def test_captured_steps_replay_as_eager_ones():
    """The whole step in a graph, replayed with new inputs in its buffers and eager work between."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    graph_loop, eager = Loop(mx, seed=3), Loop(mx, seed=3)
    names = graph_loop.inputs(0)
    held = [dev_bf16(names[0])] + [dev(x) for x in names[1:]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph_loop.step(*held)          # warm, then everything back to the start
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    fresh = Loop(mx, seed=3)
    for name in ("table", "stack", "count", "cache", "lens"):
        getattr(graph_loop, name).copy_(getattr(fresh, name))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = graph_loop.step(*held)
    for name in ("table", "stack", "count", "cache", "lens"):
        getattr(graph_loop, name).copy_(getattr(fresh, name))
    for step in range(5):
        x = graph_loop.inputs(step)
        x = [dev_bf16(x[0])] + [dev(v) for v in x[1:]]
        for h, v in zip(held, x):
            h.copy_(v)
        graph.replay()
        want = eager.step(*x)
        torch.cuda.synchronize()
        live = graph_loop.B * graph_loop.n
        assert torch.equal(got[0][:live], want[0][:live])
        for g, w in zip(got[1:], want[1:]):
            assert torch.equal(g, w), step
        assert torch.equal(graph_loop.cache, eager.cache) and torch.equal(graph_loop.table, eager.table)


def test_captured_routing_replays_as_eager():
    torch = torch_or_skip()
    mx = lib_or_fail()
    for T, E, topk in ((16, 896, 16), (3000, 64, 8)):
        x = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")
        rows = torch.zeros(1, dtype=torch.int32, device="cuda")

        def step():
            ids, w = mx.mx_moe_route(x, topk, num_rows=rows)
            return (ids, w, *mx.mx_moe_sort(ids, E))

        x.copy_(dev_bf16(W.normal_bf16((T, E), 1)))
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for i in range(4):
            x.copy_(dev_bf16(W.normal_bf16((T, E), 10 + i)))
            rows.fill_(T - 3 * i)
            graph.replay()
            want = step()
            torch.cuda.synchronize()
            for g, w in zip(got, want):
                assert torch.equal(g, w)


def test_calls_on_another_stream_and_two_at_once():
    """Each call on a stream of its own, with its own outputs and workspace, while the others run."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    x = dev_bf16(W.normal_bf16((9000, 128), 1))
    p, q, tokens, cu, kv, accept, sample = _verify_inputs([4] * 30, 5000, 2)
    v = [dev(p), dev(q), dev(tokens.astype(np.int32)), dev(cu.astype(np.int32)), dev(kv.astype(np.int32)), dev(accept), dev(sample)]
    k = dev_bf16(W.normal_bf16((700, 6, 64), 3))
    pos, slots = torch.arange(700, dtype=torch.int32, device="cuda"), torch.arange(700, device="cuda")
    freq = torch.ones(32, device="cuda") * 0.01

    def calls(stream):
        ids, w = mx.mx_moe_route(x, 8, stream=stream)
        tables = mx.mx_moe_sort(ids, 128, stream=stream)
        cache = mx._new((44, 2, KV.block_bytes(16, 64)), torch.uint8, x, stream)
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
            cache.zero_()
        y = mx.mx_kv_append(k[:, :2], k[:, 2:4], k[:, 4:], pos, slots, cache, 16, inv_freq=freq, stream=stream)
        return [ids, w, *tables, y, cache, *mx.mx_verify_drafts(*v, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = [calls(s) for s in streams]
        for _ in range(8):
            torch.full((1 << 20,), 3, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for g in got:
            for a, b in zip(g, want):
                assert torch.equal(a, b)
