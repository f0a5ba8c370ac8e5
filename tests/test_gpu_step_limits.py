"""Routing, its tables, the cache's append and the verification of drafts at sizes and inputs where
another path begins: more rows than a launch takes, offsets past 32 bits, the largest all in few
lanes, rows longer than a thread's share. Large inputs are compared with calls on a part of them, whose
results tests/test_gpu_step.py holds to the oracle, or with the oracle at some rows."""
import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O
from oracle import mx_step_oracle as S

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_step import _check_append, _check_route, _check_sort, _check_verify, _logits, _verify_inputs, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,groups,keep", [(896, 1, 1), (256, 8, 3), (1000, 5, 2), (1005, 5, 2), (64, 1, 1), (1024, 1, 1)])
@pytest.mark.parametrize("f32", [False, True])
def test_route_where_the_largest_lie_together(E, groups, keep, f32):
    """The topk largest next to each other, at strides of a lane's share, one of them far above, rising and
    falling: each way of spreading experts over lanes has its worst case among these."""
    torch_or_skip()
    mx = lib_or_fail()
    e = np.arange(E)
    base = _logits(1, E, E, f32, std=0.1)[0]
    rows = [e / 64.0 - 3, -e / 64.0, np.where(e < 20, 4.0, base), np.where(e >= E - 20, 4.0 + e / 1024.0, base)]
    for step in (2, 4, 8, 16, 64, 256):
        for at in (0, 1, step - 1):
            rows.append(np.where(e % step == at, 3.0, base))
        rows.append(np.where(e // 4 % max(1, step // 4) == 0, 2.0 - e / 1024.0, base))
    rows.append(np.where(e == E // 3, 1e30, base))
    rows.append(np.where(e % 7 == 0, -1e30, base))
    rows.append(np.where(e == E - 1, 0, -3e38))
    x = W.bf16_bits_to_f32(W.f32_to_bf16_bits(np.stack(rows).astype(np.float32)))
    bias = (np.random.default_rng(E).standard_normal(E) * 0.01).astype(np.float32)
    for topk in (1, 16, min(64, keep * E // groups)):
        for sigmoid in (False, True):
            for b in (None, bias):
                for top in (1, 2):
                    _check_route(mx, x, topk, f32, sigmoid=sigmoid, bias=b, groups=groups, topk_groups=keep, group_top=top, what=(topk, sigmoid, top))


def test_route_of_more_rows_than_a_launch_takes():
    torch = torch_or_skip()
    mx = lib_or_fail()
    T, E, topk = (1 << 22) + 77, 16, 3
    x = torch.randn((T, E), device="cuda").to(torch.bfloat16)
    rows = torch.tensor([T - 5], dtype=torch.int32, device="cuda")
    ids, w = mx.mx_moe_route(x, topk, num_rows=rows)
    for a, b in ((0, 100), ((1 << 22) - 50, T - 5)):
        i2, w2 = mx.mx_moe_route(x[a:b].contiguous(), topk)
        assert torch.equal(ids[a:b], i2) and torch.equal(w[a:b], w2)
    assert bool((ids[T - 5:] == -1).all()) and bool((w[T - 5:] == 0).all())
    assert int(ids.min()) == -1 and int(ids.max()) == E - 1


def test_route_past_32_bit_offsets():
    torch = torch_or_skip()
    mx = lib_or_fail()
    T, E, topk = 40, 1024, 8
    stride = (1 << 32) // 40 + 8                     # the last rows lie past 2^31 and 2^32 bytes and 2^31 elements
    home = torch.empty(stride * T, dtype=torch.bfloat16, device="cuda")
    x = home.as_strided((T, E), (stride, 1))
    x.copy_(torch.randn((T, E), device="cuda"))
    ids, w = mx.mx_moe_route(x, topk)
    i2, w2 = mx.mx_moe_route(x.contiguous(), topk)
    assert torch.equal(ids, i2) and torch.equal(w, w2)


@pytest.mark.parametrize("T,topk,E", [(1023, 1, 7), (1024, 1, 1024), (1025, 1, 3), (2047, 8, 896), (2048, 8, 896), (2049, 8, 896), (16384, 1, 5), (16385, 1, 5),
                                      (8192, 16, 64), (8193, 16, 64), (131072, 1, 1), (131073, 1, 1), (1 << 20, 1, 300), ((1 << 20) + 1, 1, 300), (262145, 8, 1024)])
def test_sort_at_the_borders_of_its_paths(T, topk, E):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(T)
    ids = rng.integers(0, E, (T, topk))
    if T * topk > 1 << 21:                           # the oracle's loop over experts is slow there
        flat = ids.reshape(-1)
        order = np.argsort(flat, kind="stable")
        off, tok, rows = mx.mx_moe_sort(dev(ids.astype(np.int32)), E)
        assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))]))
        assert np.array_equal(tok.cpu().numpy(), order // topk)
        want = np.empty_like(order)
        want[order] = np.arange(order.size)
        assert np.array_equal(rows.cpu().numpy().reshape(-1), want)
        return
    _check_sort(mx, ids, E)
    ids[rng.random(ids.shape) < 0.9] = -1            # nearly all of them others'
    _check_sort(mx, ids, E)


def test_append_of_more_rows_than_a_launch_takes():
    torch = torch_or_skip()
    mx = lib_or_fail()
    T, D, page = (1 << 21) + 100, 64, 1024
    rows = torch.randn((T, 3, D), device="cuda").to(torch.bfloat16)
    pages = T // page + 1
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda") + 7
    freq = dev((10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32))
    w = torch.rand(D, device="cuda") + 0.5
    cache = torch.zeros((pages, 1, KV.block_bytes(page, D)), dtype=torch.uint8, device="cuda")
    again = cache.clone()
    kw = dict(inv_freq=freq, q_weight=w, k_weight=w)
    q = mx.mx_kv_append(rows[:, :1], rows[:, 1:2], rows[:, 2:], pos, slots, cache, page, **kw)
    for a in range(0, T, 700001):
        b = min(T, a + 700001)
        q2 = mx.mx_kv_append(rows[a:b, :1], rows[a:b, 1:2], rows[a:b, 2:], pos[a:b], slots[a:b], again, page, **kw)
        assert torch.equal(q[a:b], q2)
    assert torch.equal(cache, again)


def test_append_past_32_bit_offsets():
    """Rows of a stride that takes the last past 2^32 elements, pages past 2^32 bytes."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    Hq, H, D, page, T = 2, 8, 128, 64, 40
    stride = (1 << 32) // 40 // 8 * 8 + 1024
    home = torch.empty(stride * T, dtype=torch.bfloat16, device="cuda")
    rows = home.as_strided((T, Hq + 2 * H, D), (stride, D, 1))
    bits = W.normal_bf16((T, Hq + 2 * H, D), 1)
    rows.copy_(dev_bf16(bits))
    pages = 4600 * 1000 * 1000 // (H * KV.block_bytes(page, D))
    cache = torch.zeros((pages, H, KV.block_bytes(page, D)), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    ids = np.array([pages - 1, 0, pages // 2])
    slots = ids[np.arange(T) // 16] * page + np.arange(T) % 16 + 3
    pos = np.arange(T, dtype=np.int32) * 1001
    freq = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    out = torch.empty(stride * T, dtype=torch.bfloat16, device="cuda").as_strided((T, Hq, D), (stride, D, 1))
    mx.mx_kv_append(rows[:, :Hq], rows[:, Hq:Hq + H], rows[:, Hq + H:], dev(pos), dev(slots), cache, page, inv_freq=dev(freq), q_out=out)
    y, size = S.norm_rotate(O.bf16_to_f64(bits[:, :Hq]), pos, None, 0, freq, False)
    assert np.all(np.abs(O.bf16_to_f64(host_bits(out)) - y) <= S.query_bound(y, size))
    small = np.zeros((3, H, KV.block_bytes(page, D)), np.uint8)
    S.append(small, O.bf16_to_f64(bits[:, Hq:Hq + H]), bits[:, Hq + H:], pos, np.arange(T) // 16 * page + np.arange(T) % 16 + 3, page, None, 0, freq, False)
    assert np.array_equal(cache[torch.from_numpy(ids).cuda()].cpu().numpy(), small)
    cache[torch.from_numpy(ids).cuda()] = 0
    assert int(torch.count_nonzero(cache)) == 0


@pytest.mark.parametrize("T,Hq,H,D", [(9, 7, 3, 64), (9, 9, 1, 64), (9, 5, 3, 128), (9, 3, 3, 256), (700, 9, 5, 64), (4100, 5, 3, 128)])
def test_append_leaves_what_lies_beside_its_rows(T, Hq, H, D):
    """Heads that do not fill a wave's load or a workgroup's width, in a wider row whose other columns hold
    NaN; a page's other tokens and other pages keep their bytes (test_append compares whole caches)."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    wide = torch.full((T, Hq + 2 * H + 3, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    x = dev_bf16(W.normal_bf16((T, Hq + 2 * H, D), 5))
    wide[:, 1:1 + Hq], wide[:, 2 + Hq:2 + Hq + H], wide[:, -H:] = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
    out = torch.full((T, Hq + 2, D), 3.0, dtype=torch.bfloat16, device="cuda")
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda") + 3, torch.arange(T, device="cuda") + 5
    pages = T // 16 + 2
    a = torch.full((pages, H, KV.block_bytes(16, D)), 17, dtype=torch.uint8, device="cuda")
    b = a.clone()
    w = torch.rand(D, device="cuda") + 0.5
    kw = dict(inv_freq=torch.full((D // 2,), 0.1, device="cuda"), q_weight=w, k_weight=w)
    q1 = mx.mx_kv_append(wide[:, 1:1 + Hq], wide[:, 2 + Hq:2 + Hq + H], wide[:, -H:], pos, slots, a, 16, q_out=out[:, 1:1 + Hq], **kw)
    q2 = mx.mx_kv_append(x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], pos, slots, b, 16, **kw)
    assert torch.equal(q1, q2) and torch.equal(a, b)
    assert bool((out[:, 0] == 3).all()) and bool((out[:, -1] == 3).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_norms_of_heads_near_the_largest(D):
    """What weight and scale alone would take past FP32's range, and norms below its normal numbers."""
    torch_or_skip()
    mx = lib_or_fail()
    for pairs in (False, True):
        _check_append(mx, 20, 3, 2, D, 16, std=6e37, eps=0.0, rope_scale=8.0, pairs=pairs)
        _check_append(mx, 20, 3, 2, D, 16, std=6e37, eps=1e-6, rope_scale=8.0, pairs=pairs, rot=D // 2, seed=1)


def test_append_of_zero_heads_without_eps():
    torch = torch_or_skip()
    mx = lib_or_fail()
    q = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.full((1, 2, KV.block_bytes(16, 64)), 255, dtype=torch.uint8, device="cuda")
    w = torch.ones(64, device="cuda")
    i = torch.arange(3, device="cuda")
    out = mx.mx_kv_append(q, q, q, i.int(), i, cache, 16, q_weight=w, k_weight=w, eps=0.0)
    k, v = mx.mx_kv_read(cache, i, 2, 64, 16)
    assert bool((out == 0).all()) and bool((k == 0).all()) and bool((v == 0).all())


def test_append_of_a_slot_named_twice_stays_in_its_slot():
    torch = torch_or_skip()
    mx = lib_or_fail()
    T, H, D, page = 70, 2, 64, 16
    x = dev_bf16(W.normal_bf16((T, 2 * H, D), 5))
    slots = np.arange(T, dtype=np.int64)
    slots[[9, 33, 66]] = 40
    keep = np.setdiff1d(np.arange(T), [9, 33, 66, 40])
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    kw = dict(inv_freq=torch.full((D // 2,), 0.1, device="cuda"))
    a = torch.full((6, H, KV.block_bytes(page, D)), 200, dtype=torch.uint8, device="cuda")
    b = a.clone()
    mx.mx_kv_append(None, x[:, :H], x[:, H:], pos, dev(slots), a, page, **kw)
    k = torch.from_numpy(keep).cuda()
    mx.mx_kv_append(None, x[k][:, :H], x[k][:, H:], pos[k], dev(slots[keep]), b, page, **kw)
    tok = 40 % page
    own = [KV.byte_of(kind, page, D, tok, j) for kind in ("ks", "vs") for j in range(D // 32)]
    own += [KV.byte_of(kind, page, D, tok, j, n) for kind in ("k", "v") for j in range(D // 32) for n in range(16)]
    a[40 // page][:, own] = 0
    b[40 // page][:, own] = 0
    assert torch.equal(a, b)


@pytest.mark.parametrize("V", [1023, 1024, 1025, 961, 262081, 262145, 300007, 1048579])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify_of_rows_of_every_length(V, sampled):
    """Around a wave's share, and where a thread of the second launch has more than one of them."""
    torch_or_skip()
    mx = lib_or_fail()
    rows = [3, 1] if V > 5000 else [4, 1, 2, 5]
    p, q, tokens, cu, kv, accept, sample = _verify_inputs(rows, V, V, pad_rows=1, std=3.0)
    _check_verify(mx, p, q if sampled else None, tokens, cu, kv, accept, sample)
    _check_verify(mx, p, q if sampled else None, tokens, cu, kv, accept, np.full_like(sample, 1.0), pads=(1, 1))
    _check_verify(mx, p, q if sampled else None, tokens, cu, kv, np.full_like(accept, 2.0), np.full_like(sample, 0.0), pads=(63, 5))
    one = np.zeros_like(p)
    one[:, [0, V // 2, V - 1]] = [1e-20, 1e-3, 0.5]
    for u in (0.0, 1e-10, 0.5, 0.999):
        _check_verify(mx, one, one if sampled else None, tokens, cu, kv, np.full_like(accept, 2.0), np.full_like(sample, u))


def test_verify_past_32_bit_offsets():
    torch = torch_or_skip()
    mx = lib_or_fail()
    V, T = 1000, 12
    p, q, tokens, cu, kv, accept, sample = _verify_inputs([4, 4, 3], V, 3, pad_rows=1)
    stride = (1 << 32) // 20 + 3
    args = []
    for x in (p, q):
        home = torch.empty(stride * T, device="cuda")
        rows = home.as_strided((T, V), (stride, 1))
        rows.copy_(dev(x))
        args.append(rows)
    want = S.verify(p, q, tokens, cu, kv, accept, sample)
    got = mx.mx_verify_drafts(*args, dev(tokens.astype(np.int32)), dev(cu.astype(np.int32)), dev(kv.astype(np.int32)), dev(accept), dev(sample))
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_verify_of_as_many_requests_as_a_call_takes():
    torch = torch_or_skip()
    mx = lib_or_fail()
    B, V = (1 << 16) - 2, 5
    p, q, tokens, cu, kv, accept, sample = _verify_inputs([2] * B, V, 3, pad_rows=300)
    got = mx.mx_verify_drafts(dev(p), dev(q), dev(tokens.astype(np.int32)), dev(cu.astype(np.int32)), dev(kv.astype(np.int32)), dev(accept), dev(sample))
    want = S.verify(p, q, tokens, cu, kv, accept, sample)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_draws_follow_the_target_whatever_the_draft():
    """Over a fixed grid of random numbers the tokens that a position ends up with have the target's
    shares: acceptance takes min(p, q), the rest's draws what is missing to p. With n x m numbers in the
    middle of equal cells a share is off by at most one cell a border, of which each token has two in
    each direction: 2 / n + 2 / m."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    p = np.array([0.5, 0.2, 0.2, 0.1, 0.0], np.float32)
    q = np.array([0.1, 0.2, 0.3, 0.1, 0.3], np.float32)
    n, m = 64, 64
    V, B = 5, n * m
    shares = np.zeros(V)
    for x in range(V):                                # the draft's token, with its chance
        tokens = np.full(2 * B, x, np.int32)
        accept, sample = np.repeat((np.arange(n) + 0.5) / n, m).astype(np.float32), np.tile((np.arange(m) + 0.5) / m, n).astype(np.float32)
        both = np.zeros(2 * B, np.float32)
        both[0::2] = accept
        out, acc, _ = mx.mx_verify_drafts(dev(np.tile(p, (2 * B, 1))), dev(np.tile(q, (2 * B, 1))), dev(tokens), dev(np.arange(B + 1, dtype=np.int32) * 2),
                                          torch.full((B,), 9, dtype=torch.int32, device="cuda"), dev(both), dev(sample))
        shares += q[x] * np.bincount(out.cpu().numpy()[0::2], minlength=V) / B
    assert np.all(np.abs(shares - p) <= 2 / n + 2 / m)
