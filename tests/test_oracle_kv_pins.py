"""The key/value cache oracle against hand-worked bytes, simulations by hand and invariants."""
import numpy as np

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O


def test_layout_is_a_permutation_of_the_block():
    for page, D in ((16, 64), (32, 128), (16, 256), (64, 64)):
        seen = [KV.byte_of(kind, page, D, t, j, b) for kind in ("k", "v") for t in range(page) for j in range(D // 32)
                for b in range(16)]
        seen += [KV.byte_of(kind, page, D, t, j) for kind in ("ks", "vs") for t in range(page) for j in range(D // 32)]
        assert sorted(seen) == list(range(KV.block_bytes(page, D)))


def test_layout_by_hand():
    # page 32, D = 128: 2048 B of K codes, 2048 B of V codes, 128 + 128 scale bytes
    assert KV.block_bytes(32, 128) == 4352
    assert KV.byte_of("k", 32, 128, 0, 0, 0) == 0 and KV.byte_of("k", 32, 128, 1, 0, 0) == 16
    assert KV.byte_of("k", 32, 128, 0, 1, 0) == 256 and KV.byte_of("k", 32, 128, 16, 0, 5) == 1029
    assert KV.byte_of("v", 32, 128, 0, 0, 0) == 2048 and KV.byte_of("v", 32, 128, 1, 0, 0) == 2049
    assert KV.byte_of("v", 32, 128, 0, 1, 0) == 2052 and KV.byte_of("v", 32, 128, 0, 0, 1) == 2064
    assert KV.byte_of("v", 32, 128, 4, 0, 0) == 2048 + 256 and KV.byte_of("v", 32, 128, 16, 0, 0) == 2048 + 1024
    assert KV.byte_of("ks", 32, 128, 3, 2) == 4096 + 35 and KV.byte_of("vs", 32, 128, 3, 2) == 4096 + 128 + 14


def test_write_read_round_trip_is_the_quantizer():
    rng = np.random.default_rng(0)
    T, H, D, page = 11, 2, 64, 16
    k, v = W.normal_bf16((T, H, D), seed=1), W.normal_bf16((T, H, D), seed=2, std=30.0)
    slots = rng.permutation(3 * page)[:T]
    slots[4], slots[7] = -1, 3 * page
    cache = np.zeros((3, H, KV.block_bytes(page, D)), dtype=np.uint8)
    KV.write(cache, k, v, slots, page)
    keep = [t for t in range(T) if t not in (4, 7)]
    gk, gv = KV.read(cache, slots[keep], page, D)
    for got, bits in ((gk, k), (gv, v)):
        q, s = O.quantize_mx(bits[keep].reshape(-1, D))
        assert np.array_equal(got, O.dequantize_mx(q, s).reshape(len(keep), H, D))
    # nothing but the written tokens' bytes is touched: as many nonzero scale bytes as blocks written
    assert np.count_nonzero(cache[:, :, page * D:]) == len(keep) * H * (D // 32) * 2
    qk, sk = O.quantize_mx(k.reshape(-1, D))
    whole = KV.pack(np.resize(qk, (1, H, page, D // 2)), np.resize(sk, (1, H, page, D // 32)),
                    np.resize(qk, (1, H, page, D // 2)), np.resize(sk, (1, H, page, D // 32)), page)
    rk, rv = KV.read(whole, np.arange(page), page, D)
    assert np.array_equal(rk, rv)
    assert np.array_equal(rk[3, 1], O.dequantize_mx(np.resize(qk, (H, page, D // 2))[1, 3:4],
                                                     np.resize(sk, (H, page, D // 32))[1, 3:4])[0])


def test_tables_by_hand():
    table = np.full((3, 4), 99, dtype=np.int32)
    table[0, :2] = [5, 6]      # 20 tokens
    table[1, :1] = [7]         # ended
    stack = np.array([1, 2, 3, 0], dtype=np.int32)
    cu, slots, pos, count, status, t2, s2 = KV.tables([20, 3, 0], [34, 0, 2], table, stack, 3, 16, 18)
    assert status == 0 and list(cu) == [0, 14, 14, 16]
    # page 7 comes back on top of 1, 2, 3 and goes to request 0, then 3 to request 2
    assert list(t2[0]) == [5, 6, 7, 99] and list(t2[2]) == [3, 99, 99, 99] and count == 2
    assert list(slots[:14]) == [6 * 16 + i for i in range(4, 16)] + [112, 113]
    assert list(slots[14:]) == [48, 49, -1, -1] and list(pos[14:]) == [0, 1, -1, -1]
    assert list(s2) == list(stack)
    lack = KV.tables([0, 0, 0], [64, 64, 1], table, stack, 3, 16, 200)
    assert lack[4] == 6 and not lack[0].any() and (lack[1] == -1).all() and np.array_equal(lack[5], table)
    assert KV.tables([0, 0, 0], [65, 0, 0], table, stack, 3, 16, 200)[4] == -1
    assert KV.tables([0, 0, 0], [2, 0, 0], table, stack, 3, 16, 1)[4] == -1


def test_attention_by_hand_and_invariants():
    page, D, H, G = 16, 64, 1, 2
    L, n = 19, 3
    k, v = W.normal_bf16((L, H, D), seed=3), W.normal_bf16((L, H, D), seed=4)
    cache = np.full((4, H, KV.block_bytes(page, D)), 255, dtype=np.uint8)  # unwritten bytes are NaN scales
    table = np.array([[2, 0]])
    slots = [table[0, j // page] * page + j % page for j in range(L)]
    KV.write(cache, k, v, slots, page)
    q = O.bf16_to_f64(W.normal_bf16((n + 1, G * H, D), seed=5))
    out, bound = KV.attention(q, cache, table, [0, n], [L], page, True, 0, 0.125)
    assert np.isnan(out[n]).all() and np.isfinite(out[:n]).all() and (bound[:n] > 0).all()
    kd, vd = KV.read(cache, slots, page, D)
    for i in range(n):
        for h in range(G):
            seen = L - n + i + 1
            s = [0.125 * float(np.dot(q[i, h], kd[j, 0])) for j in range(seen)]
            w = [np.exp(x - max(s)) for x in s]
            want = sum(wj * vd[j, 0] for j, wj in enumerate(w)) / sum(w)
            assert np.allclose(out[i, h], want, rtol=1e-12, atol=1e-12)
    # a window of one sees the row's own token alone
    one, _ = KV.attention(q, cache, table, [0, n], [L], page, True, 1, 0.125)
    assert np.allclose(one[:n, 0], vd[L - n:, 0], rtol=1e-12)
    # more rows than tokens: the first see nothing
    few, _ = KV.attention(q, cache, table, [0, n], [1], page, True, 0, 0.125)
    assert not few[:n - 1].any() and np.allclose(few[n - 1, 0], vd[0, 0])
    # a page outside the cache hides its tokens
    hid, _ = KV.attention(q, cache, np.array([[2, 9]]), [0, n], [L], page, False, 0, 0.125)
    sub, _ = KV.attention(q, cache, table, [0, n], [16], page, False, 0, 0.125)
    assert np.allclose(hid[:n], sub[:n], rtol=1e-12)
