"""The oracle of routing, its tables, the cache's append and the verification of drafts against
results worked out by hand."""
import math

import numpy as np

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O
from oracle import mx_step_oracle as S


def test_route_by_hand():
    l = np.log(np.array([[1, 2, 4, 1.0], [3, 3, 1, 1]]))
    ids, w = S.route(l, 2)
    assert ids.tolist() == [[2, 1], [0, 1]]
    assert np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]], rtol=1e-15)
    _, w = S.route(l, 2, renormalize=False, scale=8.0)
    assert np.allclose(w, [[4, 2], [3, 3]], rtol=1e-15)
    # a bias chooses but does not weigh
    ids, w = S.route(l[:1], 2, bias=[0, 0, -1, 0.3], renormalize=False)
    assert ids.tolist() == [[3, 1]] and np.allclose(w, [[1 / 8, 2 / 8]])
    # sigmoid of log(1), log(2), log(4): 1/2, 2/3, 4/5
    ids, w = S.route(l[:1], 3, sigmoid=True, renormalize=False)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[0.8, 2 / 3, 0.5]])


def test_route_groups_by_hand():
    p = np.array([[0.30, 0.01, 0.20, 0.19, 0.16, 0.14]])
    # two best of each group: 0.31, 0.39, 0.30; one best: 0.30, 0.20, 0.16
    assert S.route(np.log(p), 2, groups=3, topk_groups=1)[0].tolist() == [[2, 3]]
    assert S.route(np.log(p), 2, groups=3, topk_groups=1, group_top=1)[0].tolist() == [[0, 1]]
    assert S.route(np.log(p), 2, groups=3, topk_groups=2)[0].tolist() == [[0, 2]]
    assert S.route(np.log(p), 3, groups=3, topk_groups=3)[0].tolist() == [[0, 2, 3]]
    # equal groups: the lower ones
    assert S.route(np.zeros((1, 6)), 3, groups=3, topk_groups=2)[0].tolist() == [[0, 1, 2]]


def test_route_of_masked_and_padded():
    l = np.array([[-math.inf, 1, math.nan, -math.inf], [-math.inf] * 4, [math.inf, 0, math.inf, 1], [0, 0, 0, 0]])
    ids, w = S.route(l, 3, rows=3)
    assert ids.tolist() == [[1, -1, -1], [-1, -1, -1], [0, 2, 3], [-1, -1, -1]]
    assert w.tolist() == [[1, 0, 0], [0, 0, 0], [0.5, 0.5, 0], [0, 0, 0]]


def test_sort_matches_the_workloads_tables():
    ids, offsets, row_token = W.moe_routing(37, 64, 5)
    got = S.sort(ids, 64)
    assert np.array_equal(got[0], offsets) and np.array_equal(got[1], row_token)
    assert np.array_equal(got[2], W.moe_token_rows(ids))
    # a share of the experts
    off, tok, rows = S.sort([[3, 0], [-1, 4], [4, 3]], 2, first=3)
    assert off.tolist() == [0, 2, 4] and tok.tolist() == [0, 2, 1, 2, -1, -1] and rows.tolist() == [[0, -1], [-1, 2], [3, 1]]


def test_rotation_and_norm_by_hand():
    x = np.zeros((2, 1, 64))
    x[:, 0, 0], x[:, 0, 8], x[:, 0, 1], x[:, 0, 63] = 3, 4, 5, 7
    f = [math.pi / 2] + [0.0] * 7
    y, size = S.norm_rotate(x, [0, 1], None, 0, f, pairs=False)
    assert np.array_equal(y[0], x[0])
    assert np.allclose([y[1, 0, 0], y[1, 0, 8], y[1, 0, 1], y[1, 0, 63]], [-4, 3, 5, 7])
    y, _ = S.norm_rotate(x, [0, 1], None, 0, f, pairs=True, rope_scale=2.0)
    assert np.allclose([y[1, 0, 0], y[1, 0, 1], y[1, 0, 8], y[1, 0, 63]], [-10, 6, 8, 7])
    w = np.arange(64) + 1.0
    y, _ = S.norm_rotate(x, [0, 0], w, 1.0, None, pairs=False)
    r = 1 / math.sqrt((9 + 16 + 25 + 49) / 64 + 1)
    assert np.allclose(y[0, 0, [0, 1, 8, 63]], np.array([3, 10, 36, 448]) * r)


def test_append_without_norm_and_rotation_is_the_write():
    T, H, D, page = 9, 2, 64, 16
    k, v = W.normal_bf16((T, H, D), seed=1, std=5.0), W.normal_bf16((T, H, D), seed=2)
    slots = np.array([5, 40, -1, 3, 31, 48, 0, 1, 2])
    a, b = (np.zeros((3, H, KV.block_bytes(page, D)), np.uint8) for _ in range(2))
    pos = np.arange(T)
    S.append(a, O.bf16_to_f64(k), v, pos, slots, page, None, 0, None, False)
    KV.write(b, k, v, slots, page)
    assert np.array_equal(a, b)
    pos[4] = -1
    slots[4] = 47
    S.append(a, O.bf16_to_f64(k), v, pos, slots, page, None, 0, None, False)
    assert np.array_equal(a, b)


def test_verify_by_hand():
    p = np.array([[0.5, 0.25, 0.25, 0], [0.1, 0.2, 0.3, 0.4], [0, 0, 1, 0]], np.float32)
    q = np.array([[0.25, 0.75, 0, 0], [0.4, 0.2, 0.2, 0.2], [9, 9, 9, 9]], np.float32)
    run = lambda *a: [x.tolist() for x in S.verify(p, *a)]  # noqa: E731
    # token 0 (2/1 of the draft's chance) and token 0 (1/4 of it) at 0.2: both; then p's last row
    assert run(q, [7, 0, 0], [0, 3], [20], [0.99, 0.2, 0], [0.5]) == [[0, 0, 2], [2], [20]]
    # at 0.25 the second is refused: max(p - q, 0) = 0, 0, 0.1, 0.2
    assert run(q, [7, 0, 0], [0, 3], [20], [0.99, 0.25, 0], [0.3]) == [[0, 2, -1], [1], [19]]
    assert run(q, [7, 0, 0], [0, 3], [20], [0.99, 0.25, 0], [0.4]) == [[0, 3, -1], [1], [19]]
    # drafts without chance: accepted below p; p without them
    assert run(None, [7, 0, 3], [0, 3], [20], [0.49, 0.45, 0], [0.0]) == [[0, 0, -1], [1], [19]]
    assert run(None, [7, 0, 3], [0, 3], [20], [0.5, 0.4, 0], [0.5]) == [[2, -1, -1], [0], [18]]
    # requests of one row, of none, rows behind the last
    assert run(q, [7, 0, 0], [0, 1, 1], [20, 9], [0.9] * 3, [0.6, 0.5]) == [[1, -1, -1], [0, 0], [20, 9]]
    # nothing left of p: p itself; nothing of p: -1; a draft out of range
    assert run(p, [7, 3, 0], [0, 2], [20], [0.5] * 3, [0.0])[0] == [0, -1, -1]
    assert S.verify(p * 0, q, [7, 0, 0], [0, 3], [20], [0.5] * 3, [0.5])[0].tolist() == [-1, -1, -1]
    assert run(q, [7, 9, 0], [0, 2], [20], [0.0] * 3, [0.0])[:2] == [[0, -1, -1], [0]]
