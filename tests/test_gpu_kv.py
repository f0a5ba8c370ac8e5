"""GPU parity of the paged MXFP4 key/value cache (tables, write, read, attention) against the
float64 oracle (oracle/mx_kv_oracle.py).

Tables and cache bytes are compared exactly. Attention is compared within the bound that the
oracle derives from the arithmetic (KV.attention); nothing in it comes from a measured error."""
import ctypes

import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O

from gpu_util import check_gemm, dev_bf16, host_bits, lib_or_fail, torch_or_skip

pytestmark = pytest.mark.gpu


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


# ------------------------------------------------------------------------------- tables

def _request_state(rng, B, page, longest, width, spare, ended=0.2, grow=8):
    """Lengths before and after, a table and a stack that share no page."""
    old = rng.integers(0, longest + 1, B)
    new = np.minimum(old + rng.integers(0, grow + 1, B), width * page)
    new = np.where(rng.random(B) < ended, rng.integers(0, old + 1), new)
    held = -(-old // page)
    pages = int(held.sum()) + spare
    ids = rng.permutation(pages).astype(np.int32)
    table = rng.integers(-5, pages, (B, width)).astype(np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    stack = np.full(pages + 3, -7, dtype=np.int32)
    stack[:spare] = ids[at:]
    return old.astype(np.int32), new.astype(np.int32), table, stack, spare


def _check_tables(mx, old, new, table, stack, count, page, rows, alias=False):
    import torch
    want = KV.tables(old, new, table, stack, count, page, rows)
    t, s = dev(table), dev(stack)
    c = torch.tensor([count, 12345], dtype=torch.int32, device="cuda")
    for again in range(1 if alias else 2):  # the same arguments give the same result
        cu, slots, pos, after, status = mx.mx_kv_tables(dev(old), dev(new), t, s, c[:1], page, rows,
                                                        free_count_out=c[:1] if alias else None)
        got = [x.cpu().numpy() for x in (cu, slots, pos)] + [int(after[0]), int(status[0]), t.cpu().numpy(), s.cpu().numpy()]
        for name, g, w in zip(("cu_q", "slots", "positions", "count", "status", "table", "stack"), got, want):
            assert np.array_equal(g, w), (name, again)
    assert int(c[1]) == 12345
    return want


@pytest.mark.parametrize("B,page,longest,width,grow,pad", [
    (1, 16, 0, 4, 1, 0), (1, 16, 40, 8, 3, 5), (7, 32, 200, 12, 40, 1), (96, 16, 600, 64, 1, 0),
    (1024, 16, 100, 12, 2, 9), (1025, 16, 60, 8, 4, 3), (3000, 64, 500, 16, 5, 0), (20, 128, 900, 200, 2000, 7),
    (2, 1024, 5000, 40, 9000, 0)])
def test_tables_match_a_plain_stack(B, page, longest, width, grow, pad):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(B * 1000 + page)
    for alias in (False, True):
        old, new, table, stack, count = _request_state(rng, B, page, longest, width, 4 + B * (2 + grow // page), grow=grow)
        rows = int(np.maximum(new - old, 0).sum()) + pad
        want = _check_tables(mx, old, new, table, stack, count, page, rows, alias)
        assert want[4] == 0


@pytest.mark.parametrize("B", [5, 2000])
def test_tables_refuse_on_the_device_and_change_nothing(B):
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(B)
    old, new, table, stack, count = _request_state(rng, B, 16, 100, 20, 3 * B, ended=0.0)
    rows = int((new - old).sum())
    new[0], old[0] = 300, 1                              # one request grows by 18 pages or so
    rows = int(np.maximum(new - old, 0).sum())
    taken = int((-(-new // 16) + (-old // 16)).sum())
    assert _check_tables(mx, old, new, table, stack, taken, 16, rows)[4] == 0           # just enough
    assert _check_tables(mx, old, new, table, stack, taken - 1, 16, rows)[4] == 1       # one page short
    assert _check_tables(mx, old, new, table, stack, 0, 16, rows)[4] == taken
    assert _check_tables(mx, old, new, table, stack, count, 16, rows - 1)[4] == -1      # rows do not fit
    assert _check_tables(mx, old, new, table, stack, len(stack) + 1, 16, rows)[4] == -1
    assert _check_tables(mx, old, new, table, stack, -1, 16, rows)[4] == -1
    for b, o, n in ((B - 1, -1, 3), (0, 5, -2), (B // 2, 0, 20 * 16 + 1), (B // 2, 2 ** 31 - 1, 0), (1, 0, 2 ** 31 - 1)):
        o2, n2 = old.copy(), new.copy()
        o2[b], n2[b] = o, n
        assert _check_tables(mx, o2, n2, table, stack, count, 16, rows + 20)[4] == -1
    # pages given back that do not fit the stack
    assert _check_tables(mx, old, np.zeros_like(new), table, stack[:count], count, 16, rows)[4] == -1
    # sums past 31 bits are refused, not wrapped
    wide = np.full(B, 2 ** 31 - 1024, dtype=np.int32)
    one = np.zeros((B, 1), dtype=np.int32)
    got = mx.mx_kv_tables(dev(np.zeros(B, np.int32)), dev(wide), dev(one), dev(stack), dev(np.array([3], np.int32)), 1024, 8)
    assert int(got[4][0]) == -1 and int(got[3][0]) == 3


def test_tables_of_nothing():
    torch = torch_or_skip()
    mx = lib_or_fail()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    c = torch.tensor([2], dtype=torch.int32, device="cuda")
    cu, slots, pos, after, status = mx.mx_kv_tables(e, e, torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                                                    torch.tensor([8, 9], dtype=torch.int32, device="cuda"), c, 16, 3)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3
    assert after.tolist() == [2] and status.tolist() == [0]


# ------------------------------------------------------------------------------- write, read

@pytest.mark.parametrize("T,H,D,page,layout", [
    (1, 1, 64, 16, "dense"), (5, 3, 64, 16, "fused"), (64, 8, 128, 32, "fused"), (131, 2, 256, 64, "dense"),
    (37, 5, 128, 1024, "dense"), (200, 1, 64, 16, "fused"), (66, 7, 64, 128, "expanded")])
@pytest.mark.parametrize("order", ["random", "run"])
def test_write_bytes_match_the_oracle(T, H, D, page, layout, order):
    torch = torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 2
    bits = W.normal_bf16((T, 3 * H, D), seed=T, std=4.0)
    bits[T // 2, :, :32] = 0                              # an all-zero block
    bits[T // 3, :, 32:64] = 0x8000                       # negative zeros
    bits[0, :, 0] = 0x7F7F                                # bf16's largest
    bits[T - 1, 0, 33] = 0x0001                           # and its least subnormal
    if layout == "expanded":
        bits = np.broadcast_to(bits[:1], bits.shape).copy()
    wide = dev_bf16(bits)
    if layout == "expanded":
        wide = wide[:1].expand(T, -1, -1)
    k, v = wide[:, H:2 * H], wide[:, 2 * H:]
    if layout == "dense":
        k, v = k.contiguous(), v.contiguous()
    slots = rng.permutation(pages * page)[:T] if order == "random" else np.arange(T) + page // 3
    slots = slots.astype(np.int64)
    if T > 4:
        slots[2], slots[4], slots[3] = -1, pages * page, 1 << 40
    start = rng.integers(0, 256, (pages, H, KV.block_bytes(page, D)), dtype=np.uint8)
    cache = dev(start)
    mx.mx_kv_write(k, v, dev(slots), cache, page)
    want = start.copy()
    KV.write(want, bits[:, H:2 * H], bits[:, 2 * H:], slots, page)
    assert np.array_equal(cache.cpu().numpy(), want)
    # and what the cache stands for
    kept = np.flatnonzero((slots >= 0) & (slots < pages * page))
    kr = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    vr = kr.clone()
    mx.mx_kv_read(cache, dev(slots), H, D, page, k_out=kr, v_out=vr)
    wk, wv = KV.read(want, slots[kept], page, D)
    for got, exact in ((kr, wk), (vr, wv)):
        g = O.bf16_to_f64(host_bits(got))
        # blocks below bf16's range (scale 2^-127 times 0.5) may lose their last bit
        assert np.all(np.abs(g[kept] - exact) <= 2.0 ** -127)
        gone = np.setdiff1d(np.arange(T), kept)
        assert np.all(g[gone] == 7.0)


def test_write_of_a_slot_named_twice_stays_in_its_slot():
    """The documentation leaves open whose bytes it holds; no other slot's byte changes."""
    torch_or_skip()
    mx = lib_or_fail()
    T, H, D, page = 70, 2, 64, 16
    k, v = W.normal_bf16((T, H, D), seed=5), W.normal_bf16((T, H, D), seed=6)
    slots = np.arange(T, dtype=np.int64)
    slots[[9, 33, 66]] = 40                                # and 40 itself
    start = np.random.default_rng(7).integers(0, 256, (6, H, KV.block_bytes(page, D)), dtype=np.uint8)
    cache = dev(start)
    mx.mx_kv_write(dev_bf16(k), dev_bf16(v), dev(slots), cache, page)
    got = cache.cpu().numpy()
    keep = np.setdiff1d(np.arange(T), [9, 33, 66, 40])
    want = start.copy()
    KV.write(want, k[keep], v[keep], slots[keep], page)
    own = np.zeros(start.shape[2], dtype=bool)             # the bytes of slot 40 in its page
    tok = 40 % page
    for j in range(D // 32):
        own[[KV.byte_of(kind, page, D, tok, j) for kind in ("ks", "vs")]] = True
        for b in range(16):
            own[[KV.byte_of(kind, page, D, tok, j, b) for kind in ("k", "v")]] = True
    same = got == want
    same[40 // page, :, own] = True
    assert same.all()


def test_cache_past_32_bit_offsets():
    """A cache of 4.6 GB: pages whose bytes lie past 2^31 and 2^32."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    H, D, page = 8, 128, 64
    pages = 4600 * 1000 * 1000 // (H * KV.block_bytes(page, D))
    cache = torch.zeros((pages, H, KV.block_bytes(page, D)), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    L = 200
    k, v = W.normal_bf16((L, H, D), seed=1), W.normal_bf16((L, H, D), seed=2)
    ids = np.array([[pages - 1, 3, pages // 2, pages - 2]], dtype=np.int32)
    pos = np.arange(L)
    slots = ids[0, pos // page].astype(np.int64) * page + pos % page
    mx.mx_kv_write(dev_bf16(k), dev_bf16(v), dev(slots), cache, page)
    kr, vr = mx.mx_kv_read(cache, dev(slots), H, D, page)
    small = np.zeros((4, H, KV.block_bytes(page, D)), dtype=np.uint8)
    KV.write(small, k, v, pos, page)
    wk, wv = KV.read(small, pos, page, D)
    assert np.array_equal(O.bf16_to_f64(host_bits(kr)), wk) and np.array_equal(O.bf16_to_f64(host_bits(vr)), wv)
    q = W.normal_bf16((5, 16, D), seed=3)
    out = mx.mx_kv_attention(dev_bf16(q), cache, dev(ids), dev(np.array([0, 5], np.int32)), dev(np.array([L], np.int32)), H, page)
    exact, bound = KV.attention(O.bf16_to_f64(q), small, np.arange(4)[None], [0, 5], [L], page, True, 0, D ** -0.5)
    _close(host_bits(out), exact, bound, "past 32 bits")


# ------------------------------------------------------------------------------- attention

def _close(bits, exact, bound, what):
    got = O.bf16_to_f64(bits)
    bad = ~(np.abs(got - exact) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first at {i}: got {got[i]!r} exact {exact[i]!r} "
                             f"bound {bound[i]!r}")


class Case:
    """A cache with requests in it, on the host and on the device."""

    def __init__(self, D, H, G, page, q_lens, kv_lens, seed=0, q_std=1.5, k_std=1.0, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.D, self.H, self.G, self.page = D, H, G, page
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        each = [-(-n // page) for n in kv_lens]
        used = sum(each)
        self.pages = used + 3
        n = self.pages * H * page
        qk, sk = O.quantize_mx(W.normal_bf16((n, D), seed=seed + 1, std=k_std))
        qv, sv = O.quantize_mx(W.normal_bf16((n, D), seed=seed + 2))
        sh = (self.pages, H, page)
        self.cache = KV.pack(qk.reshape(*sh, -1), sk.reshape(*sh, -1), qv.reshape(*sh, -1), sv.reshape(*sh, -1), page)
        ids = rng.permutation(self.pages).astype(np.int32)
        width = max(each + [1]) + 1
        self.table = np.full((len(kv_lens), width), -1, dtype=np.int32)
        at = 0
        for b, e in enumerate(each):
            self.table[b, :e] = ids[at:at + e]
            at += e
        # bytes past a request's end were never written: NaN scales and all-ones codes
        m, P = D // 32, page
        for b, L in enumerate(kv_lens):
            for tok in range(L % P, P) if L % P else ():
                blk = self.cache[self.table[b, L // P]]
                for j in range(m):
                    blk[:, KV.byte_of("ks", P, D, tok, j)] = 255
                    blk[:, KV.byte_of("vs", P, D, tok, j)] = 255
                    for i in range(16):
                        blk[:, KV.byte_of("k", P, D, tok, j, i)] = 255
                        blk[:, KV.byte_of("v", P, D, tok, j, i)] = 255
        for p in ids[used:]:
            self.cache[p] = 255
        self.cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.T = int(self.cu[-1]) + extra_rows
        self.q = W.normal_bf16((self.T, H * G, D), seed=seed + 3, std=q_std)

    def exact(self, causal=True, window=0, scale=None):
        return KV.attention(O.bf16_to_f64(self.q), self.cache, self.table, self.cu, self.kv_lens, self.page, causal, window,
                            self.D ** -0.5 if scale is None else scale)

    def args(self):
        return (dev(self.cache), dev(self.table), dev(self.cu), dev(np.array(self.kv_lens, np.int32)), self.H, self.page)

    def check(self, mx, causal=True, window=0, scale=None, what="", **kw):
        import torch
        exact, bound = self.exact(causal, window, scale)
        n = int(self.cu[-1])
        out = torch.full((self.T, self.H * self.G, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        kw.setdefault("max_q", max(self.q_lens + [1]))
        kw.setdefault("max_kv", max(self.kv_lens + [1]))
        q = kw.pop("q", None)
        mx.mx_kv_attention(dev_bf16(self.q) if q is None else q, *self.args(), causal=causal, window=window, scale=scale, out=out, **kw)
        bits = host_bits(out)
        _close(bits[:n], exact[:n], bound[:n], what)
        assert np.all(O.bf16_to_f64(bits[n:]) == 7.0), "rows behind the last request were written"
        return bits


# decoding and drafts: D, H, G, page, q, kv lengths
FEW = [
    (64, 1, 1, 16, 1, [1]), (128, 1, 1, 16, 1, [2, 15, 16, 17]), (256, 1, 1, 16, 1, [31, 33]),
    (64, 2, 3, 32, 1, [63, 64, 65, 0, 129]), (128, 2, 8, 16, 1, [255, 256, 257, 1, 700]), (256, 2, 4, 64, 1, [500, 12]),
    (128, 1, 16, 128, 1, [1000, 77]), (128, 1, 12, 16, 1, [300]), (64, 1, 5, 16, 3, [40, 2, 0, 65]),
    (128, 2, 2, 16, 8, [129, 8, 7, 513]), (256, 1, 3, 32, 5, [90, 5]), (128, 3, 1, 64, 4, [1500, 3]),
    (128, 1, 20, 16, 1, [50, 1000]), (64, 1, 32, 16, 1, [333]), (128, 1, 4, 1024, 2, [2100, 1025]),
]


@pytest.mark.parametrize("D,H,G,page,q,kv", FEW)
def test_attention_of_few_rows(D, H, G, page, q, kv):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, page, [q] * len(kv), kv, seed=D + H + G + page + q, extra_rows=2)
    c.check(mx, what="causal")
    c.check(mx, causal=False, what="all")
    c.check(mx, workspace=False, what="no workspace")


@pytest.mark.parametrize("B", [257, 700])
def test_attention_of_many_requests(B):
    """More requests than a workgroup has threads, ragged, some empty, alone and beside a chunk."""
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 90, B)
    kv[B // 2] = 5000
    c = Case(64, 1, 2, 16, [1] * B, kv, seed=B)
    c.check(mx, what="decode")
    c.check(mx, workspace=False, what="no workspace")
    q = rng.integers(0, 3, B)
    q[B - 1], kv[B - 1] = 60, 200
    c = Case(64, 1, 2, 16, q, kv, seed=B + 1, extra_rows=1)
    c.check(mx, what="mixed")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q,max_kv", [(1, 64), (1, 100000), (150, 400)])
def test_attention_of_many_requests_of_several_tiles(D, max_q, max_kv):
    """Row tiles past each request's first, searched for among more requests than a wave has lanes, in
    each kernel: with a hint of one row the few-rows kernel takes them all, whole and shared."""
    torch_or_skip()
    mx = lib_or_fail()
    rng = np.random.default_rng(D + max_q)
    B = 131
    kv = rng.integers(0, 120, B)
    q = np.minimum(rng.integers(0, 3, B) * rng.integers(0, 20, B), 17)
    kv[3], q[3] = 400, 150  # several tiles of 128 rows
    kv[B - 1], q[B - 1] = 333, 90
    c = Case(D, 2, 2, 16, q, kv, seed=B + D, extra_rows=5)
    c.check(mx, max_q=max_q, max_kv=max_kv, what=f"hints {max_q} {max_kv}")


# prompts and chunks: D, H, G, page, row counts, kv lengths
MANY = [
    (64, 1, 1, 16, [33], [33]), (128, 1, 1, 16, [64, 65, 1], [64, 65, 100]), (256, 1, 1, 16, [40], [300]),
    (128, 2, 4, 16, [17, 0, 130, 5], [17, 40, 500, 5]), (64, 2, 3, 64, [127, 128, 129], [127, 200, 513]),
    (128, 1, 8, 32, [300, 2], [301, 600]), (256, 2, 2, 128, [70, 150], [70, 151]), (128, 1, 16, 16, [40], [1030]),
    (128, 1, 5, 16, [50, 3], [30, 2]), (64, 1, 40, 16, [1, 2], [100, 260]), (64, 1, 1, 16, [133], [133]),
    (128, 1, 1, 16, [129, 200, 1], [129, 200, 100]), (256, 1, 1, 16, [140], [300]), (64, 2, 40, 16, [3, 4, 5], [100, 260, 5]),
]


@pytest.mark.parametrize("D,H,G,page,q,kv", MANY)
def test_attention_of_many_rows(D, H, G, page, q, kv):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, page, q, kv, seed=D + H + G + page + sum(q), extra_rows=3)
    c.check(mx, what="causal")
    c.check(mx, causal=False, what="all")
    c.check(mx, workspace=False, what="no workspace")


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 100, 1000, 2 ** 31 - 1, 2 ** 33])
@pytest.mark.parametrize("D,q,kv", [(128, [1, 1, 4], [200, 17, 600]), (128, [70, 1, 33], [200, 1, 333]), (256, [40], [40]),
                                    (64, [1, 90], [700, 128]), (128, [170, 1, 33], [200, 1, 333]), (256, [140], [140]),
                                    (64, [1, 190], [700, 228])])
def test_attention_window(window, D, q, kv):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, 1, 3, 16, q, kv, seed=window % 1000 + D)
    # pages that no row sees may have been given away: their entries name no page
    for b, (n, L) in enumerate(zip(q, kv)):
        first = max(0, L - n - window + 1) // 16
        c.table[b, :first] = 1 << 30
    c.check(mx, window=window, what=f"window {window}")


def test_attention_long_and_split():
    """One request of 131072 tokens and a short one: the tokens are split over the chip."""
    torch_or_skip()
    mx = lib_or_fail()
    for D, G in ((64, 2), (128, 1)):
        c = Case(D, 1, G, 128, [1, 1], [131072, 70], seed=D)
        c.check(mx, what="decode")
    c = Case(128, 1, 2, 64, [40, 2], [20011, 20], seed=5)
    c.check(mx, what="chunk")


@pytest.mark.parametrize("max_q,max_kv", [(1, 1), (1, 100000), (4096, 1), (4096, 100000), (7, 60)])
def test_attention_hints_change_no_result(max_q, max_kv):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(128, 2, 4, 16, [1, 50, 0, 7, 1, 1], [900, 77, 30, 7, 1, 0], seed=9, extra_rows=1)
    c.check(mx, max_q=max_q, max_kv=max_kv, what=f"hints {max_q} {max_kv}")


def test_attention_bad_pages_hide_their_tokens():
    torch_or_skip()
    mx = lib_or_fail()
    for q in ([1, 2], [60, 3]):
        c = Case(128, 1, 2, 16, q, [200, 90], seed=11)
        c.table[0, 0], c.table[0, 5], c.table[1, 2] = c.pages, -1, 2 ** 31 - 1
        c.table[0, 11] = -(2 ** 31)
        c.table[1, 5] = c.pages + 7                        # the last, ragged page
        c.check(mx, what="bad pages")
        c.table[:] = -1
        assert not c.check(mx, what="no page at all")[:sum(q)].any()


def test_attention_garbage_lengths_stay_in_bounds():
    """Lengths and offsets outside their ranges are clamped: nothing outside the buffers is touched."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    c = Case(128, 1, 4, 16, [1, 30, 2], [90, 90, 20], seed=12)
    cache, table, cu, kv, H, page = c.args()
    T = c.T
    for cu_bad, kv_bad in (([0, 1, 31, 9999], [90, 90, 20]), ([-5, 1, 31, 33], [90, 2 ** 31 - 1, -7]), ([0, 31, 1, 33], [90] * 3),
                           ([2 ** 31 - 1] * 4, [1] * 3), ([-2 ** 31] * 4, [1] * 3)):
        guard = torch.full((T + 2, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.mx_kv_attention(dev_bf16(c.q), cache, table, dev(np.array(cu_bad, np.int32)), dev(np.array(kv_bad, np.int32)), H, page,
                           out=guard[1:T + 1], max_q=30, max_kv=90)
        torch.cuda.synchronize()
        assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())


def test_attention_extreme_values():
    """Scores of +-thousands, one weight that is all the sum, V blocks at both ends of the scale's
    range, and queries whose elements differ by 2^40."""
    torch_or_skip()
    mx = lib_or_fail()
    for q in ([1], [40]):
        c = Case(128, 1, 2, 16, q, [150], seed=13, q_std=60.0, k_std=20.0)
        c.check(mx, what="large scores")
        bits = c.q.copy()
        f = O.bf16_to_f64(bits)
        f[..., ::7] *= 2.0 ** -40
        c.q = W.f32_to_bf16_bits(f.astype(np.float32))
        c.check(mx, what="spread queries")
        c.q = W.f32_to_bf16_bits((O.bf16_to_f64(bits) * 2.0 ** 90).astype(np.float32))
        c.check(mx, scale=2.0 ** -100, what="large queries")
        c.q = W.f32_to_bf16_bits((O.bf16_to_f64(bits) * 2.0 ** -100).astype(np.float32))
        c.check(mx, scale=2.0 ** 90, what="tiny queries")
        c.q[:] = 0
        c.check(mx, what="zero queries")
    c = Case(128, 1, 2, 16, [3], [150], seed=14)
    P, D = c.page, c.D
    for tok in range(0, 150, 3):
        blk = c.cache[c.table[0, tok // P]]
        blk[:, KV.byte_of("vs", P, D, tok % P, 1)] = 127 + 100
        blk[:, KV.byte_of("vs", P, D, tok % P, 2)] = 10
    c.check(mx, what="V scales")


def test_attention_of_shared_pages():
    """Requests that share the pages of a common beginning, and one page twice in a request."""
    torch_or_skip()
    mx = lib_or_fail()
    for q in ([1, 1, 2], [40, 1, 50]):
        c = Case(128, 2, 2, 16, q, [100, 90, 120], seed=21)
        c.table[1, :4] = c.table[0, :4]
        c.table[2, 3] = c.table[2, 1]
        c.check(mx, what="shared")


def test_attention_calls_at_the_same_time():
    """Two streams, each with its own workspace and output, many calls in flight."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    cases = [Case(128, 2, 4, 16, [1, 1, 1], [3000, 1700, 40], seed=22), Case(128, 1, 2, 16, [100, 3], [2500, 800], seed=23)]
    want = [c.check(mx) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    inputs = [(dev_bf16(c.q), c.args(), dict(max_q=max(c.q_lens), max_kv=max(c.kv_lens))) for c in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(12):
        for i, (q, args, kw) in enumerate(inputs):
            outs[i].append(mx.mx_kv_attention(q, *args, stream=streams[i], **kw))
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(np.array_equal(host_bits(o), w) for o in got)


def test_attention_strided_rows_and_output():
    torch = torch_or_skip()
    mx = lib_or_fail()
    for q in ([1, 2, 3], [60, 1]):
        kv = [100 + n for n in q]
        c = Case(128, 2, 2, 16, q, kv, seed=15)
        wide = torch.zeros((c.T, 8, 128), dtype=torch.bfloat16, device="cuda")
        wide[:, :4] = dev_bf16(c.q)
        exact, bound = c.exact()
        home = torch.full((c.T, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.mx_kv_attention(wide[:, :4], *c.args(), out=home[:, 1:5], max_q=max(q), max_kv=max(kv))
        _close(host_bits(home[:, 1:5]), exact, bound, "strided")
        assert bool((home[:, 0] == 7).all()) and bool((home[:, 5] == 7).all())


def test_attention_is_reproducible_and_ignores_the_batch():
    """Bit for bit the same again, and whatever stands in unseen bytes."""
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(128, 2, 4, 16, [1, 4, 40], [900, 333, 200], seed=16)
    first = c.check(mx)
    assert np.array_equal(first, c.check(mx))
    c.cache = np.where(c.cache == 255, 0, c.cache)
    changed = Case(128, 2, 4, 16, [1, 4, 40], [900, 333, 200], seed=16)
    used = {int(p) for row, L in zip(changed.table, changed.kv_lens) for p in row[:-(-L // 16)]}
    for p in range(changed.pages):
        if p not in used:
            changed.cache[p] = 0
    assert np.array_equal(first, changed.check(mx))


def test_attention_on_another_stream_and_in_graphs():
    """A side stream, and two captured graphs with a workspace each, replayed between eager calls."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    cases = [Case(128, 2, 4, 16, [1, 1], [2000, 900], seed=17), Case(128, 1, 2, 16, [50], [700], seed=18)]
    want = [c.check(mx) for c in cases]
    side = torch.cuda.Stream()
    graphs = []
    for c, w in zip(cases, want):
        q, args = dev_bf16(c.q), c.args()
        kw = dict(max_q=max(c.q_lens), max_kv=max(c.kv_lens))
        torch.cuda.synchronize()
        out = mx.mx_kv_attention(q, *args, stream=side, **kw)
        side.synchronize()
        assert np.array_equal(host_bits(out), w)
        B, T = len(c.kv_lens), c.T
        nbytes = mx.mx_kv_attention_workspace_bytes(B, T, c.H * c.G, c.H, c.D, kw["max_q"], kw["max_kv"])
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.mx_kv_attention(q, *args, out=out, workspace=ws, **kw)
        graphs.append((g, out, q, args, ws))
    for _ in range(4):
        for (g, out, *_), w, c in zip(graphs, want, cases):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(host_bits(out), w)
            assert np.array_equal(c.check(mx), w)


# ------------------------------------------------------------------------------- a run of them

def test_serving_steps_from_projection_to_projection():
    """The layer's path as a serving loop runs it: the fused QKV projection (mx_a4w4_gemm), tables,
    write, attention, the output projection; a prompt step, then decoding steps captured once into a
    graph and replayed, one request ending on the way. Every step's parts are checked against the
    oracle from the step's own inputs."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    B, H, G, D, page, K = 3, 2, 4, 128, 16, 512
    Hq, N = H * G, (H * G + 2 * H) * D
    pages, width, rows_max = 24, 12, 64
    wqkv = mx.mx_prepare_weight(dev_bf16(W.dense_weight(N, K, seed=71)))
    wo_bits = W.dense_weight(256, Hq * D, seed=72)
    wo = mx.mx_prepare_weight(dev_bf16(wo_bits))
    i32 = dict(dtype=torch.int32, device="cuda")
    table, stack = torch.full((B, width), -1, **i32), torch.arange(pages, **i32)
    count, old, new = torch.tensor([pages], **i32), torch.zeros(B, **i32), torch.zeros(B, **i32)
    cu, slots, pos = torch.zeros(B + 1, **i32), torch.zeros(rows_max, dtype=torch.int64, device="cuda"), torch.zeros(rows_max, **i32)
    status = torch.zeros(1, **i32)
    cache = torch.full((mx.mx_kv_cache_bytes(pages, page, H, D),), 255, dtype=torch.uint8, device="cuda")
    x = torch.zeros((rows_max, K), dtype=torch.bfloat16, device="cuda")
    host = {"table": table.cpu().numpy(), "stack": stack.cpu().numpy(), "count": pages,
            "cache": cache.cpu().numpy().reshape(pages, H, -1)}

    def step(qkv, out, y):
        mx.mx_kv_tables(old, new, table, stack, count, page, rows_max, cu_q=cu, slots=slots, positions=pos, free_count_out=count,
                        status=status)
        mx.mx_a4w4_gemm(x, wqkv, N, out=qkv, workspace=False)
        heads = qkv.view(rows_max, -1, D)
        mx.mx_kv_write(heads[:, Hq:Hq + H], heads[:, Hq + H:], slots, cache, page)
        mx.mx_kv_attention(heads[:, :Hq], cache, table, cu, new, H, page, out=out, max_q=rows_max, max_kv=width * page, workspace=False)
        mx.mx_a4w4_gemm(out.view(rows_max, Hq * D), wo, 256, out=y, workspace=False)

    def buffers():
        bf = dict(dtype=torch.bfloat16, device="cuda")
        return torch.zeros((rows_max, N), **bf), torch.zeros((rows_max, Hq, D), **bf), torch.zeros((rows_max, 256), **bf)

    def check(lens0, lens1, qkv, out, y):
        torch.cuda.synchronize()
        wcu, wslots, wpos, host["count"], st, host["table"], host["stack"] = KV.tables(
            lens0, lens1, host["table"], host["stack"], host["count"], page, rows_max)
        assert st == 0 and int(status[0]) == 0 and int(count[0]) == host["count"]
        for got, want in ((cu, wcu), (slots, wslots), (pos, wpos), (table, host["table"]), (stack, host["stack"])):
            assert np.array_equal(got.cpu().numpy(), want)
        bits = host_bits(qkv).reshape(rows_max, -1, D)
        KV.write(host["cache"], bits[:, Hq:Hq + H], bits[:, Hq + H:], wslots, page)
        assert np.array_equal(cache.cpu().numpy(), host["cache"].reshape(-1))
        n = int(wcu[-1])
        exact, bound = KV.attention(O.bf16_to_f64(bits[:, :Hq]), host["cache"], host["table"], wcu, lens1, page, True, 0, D ** -0.5)
        ob = host_bits(out)
        _close(ob[:n], exact[:n], bound[:n], "step")
        check_gemm(host_bits(y)[:n], O.gemm_ref(ob[:n].reshape(n, Hq * D), wo_bits), what="output projection")

    lens = [[0, 0, 0], [20, 33, 5], [21, 34, 6], [22, 35, 7], [23, 0, 8], [24, 0, 9]]
    bufs = buffers()

    def feed(i):
        old.copy_(torch.tensor(lens[i - 1], **i32))
        new.copy_(torch.tensor(lens[i], **i32))
        x.copy_(dev_bf16(W.normal_bf16((rows_max, K), seed=80 + i)))

    feed(1)
    step(*bufs)
    check(lens[0], lens[1], *bufs)
    # warm up on a copy of the state's inputs is not needed: nothing in the step allocates or compiles
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(*bufs)
    for i in range(2, len(lens)):
        feed(i)
        g.replay()
        check(lens[i - 1], lens[i], *bufs)
