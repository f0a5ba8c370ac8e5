"""CPU oracle for the paged MXFP4 key/value cache: its layout, its tables and its attention.

TEST INFRASTRUCTURE ONLY. The test suite is the only caller; the product library never
imports, links or runs anything here. Everything is NumPy in float64 or integers, written
from the definitions in include/mx.h.
"""
from __future__ import annotations

import numpy as np

from . import mx_oracle as O


def block_bytes(page: int, D: int) -> int:
    return page * D * 17 // 16


# ------------------------------------------------------------------------------- the layout

def byte_of(kind: str, page: int, D: int, tok: int, j: int, b: int = 0) -> int:
    """Offset in a (page, head) block of byte b of scale block j of token tok: kind "k" or "v"
    for codes, "ks" or "vs" for the scale byte. One formula per line of the header's table."""
    m = D // 32
    tile, r = divmod(tok, 16)
    if kind == "k":
        return ((tile * m + j) * 16 + r) * 16 + b
    if kind == "v":
        return page * D // 2 + (((tile * 4 + r // 4) * 16 + b) * m + j) * 4 + r % 4
    if kind == "ks":
        return page * D + (tile * m + j) * 16 + r
    if kind == "vs":
        return page * D + page * m + tok * m + j
    raise ValueError(kind)


def _maps(page: int, D: int):
    """Index arrays into a block: codes [page, m, 16] for k and v, scales [page, m] for each."""
    tok, j, b = np.meshgrid(np.arange(page), np.arange(D // 32), np.arange(16), indexing="ij")
    f = np.vectorize(byte_of, excluded=["kind", "page", "D"], otypes=[np.int64])
    return (f("k", page, D, tok, j, b), f("v", page, D, tok, j, b), f("ks", page, D, tok[..., 0], j[..., 0]),
            f("vs", page, D, tok[..., 0], j[..., 0]))


def write(cache: np.ndarray, k_bits: np.ndarray, v_bits: np.ndarray, slots, page: int) -> None:
    """Quantize bf16 rows [T, H, D] into cache uint8 [pages, H, block]; slots outside are skipped."""
    T, H, D = k_bits.shape
    mk, mv, mks, mvs = _maps(page, D)
    for bits, mc, ms in ((k_bits, mk, mks), (v_bits, mv, mvs)):
        q, s = O.quantize_mx(bits.reshape(T * H, D))
        q, s = q.reshape(T, H, D // 32, 16), s.reshape(T, H, D // 32)
        for t, slot in enumerate(slots):
            if 0 <= slot < cache.shape[0] * page:
                p, tok = divmod(int(slot), page)
                for h in range(H):
                    cache[p, h, mc[tok]] = q[t, h]
                    cache[p, h, ms[tok]] = s[t, h]


def pack(qk, sk, qv, sv, page: int) -> np.ndarray:
    """cache [pages, H, block] of payloads [pages, H, page, D/2] and scales [pages, H, page, m]."""
    pages, H, _, half = qk.shape
    D = 2 * half
    m = D // 32
    out = np.empty((pages, H, block_bytes(page, D)), dtype=np.uint8)
    mk, mv, mks, mvs = _maps(page, D)
    out[..., mk.reshape(-1)] = qk.reshape(pages, H, page * half)
    out[..., mv.reshape(-1)] = qv.reshape(pages, H, page * half)
    out[..., mks.reshape(-1)] = sk.reshape(pages, H, page * m)
    out[..., mvs.reshape(-1)] = sv.reshape(pages, H, page * m)
    return out


def read(cache: np.ndarray, slots, page: int, D: int):
    """float64 (k, v) [T, H, D] at `slots` (all of them inside the cache)."""
    H = cache.shape[1]
    mk, mv, mks, mvs = _maps(page, D)
    out = []
    for mc, ms in ((mk, mks), (mv, mvs)):
        rows = []
        for slot in slots:
            p, tok = divmod(int(slot), page)
            q = cache[p][:, mc[tok].reshape(-1)]
            rows.append(O.dequantize_mx(q, cache[p][:, ms[tok]]))
        out.append(np.stack(rows) if rows else np.zeros((0, H, D)))
    return tuple(out)


# ------------------------------------------------------------------------------- the tables

def tables(old, new, table, stack, count, page, rows):
    """Block tables and slots by a plain stack: (cu_q, slots, positions, count, status, table,
    stack), arrays copied."""
    table, stack = np.array(table, dtype=np.int32), np.array(stack, dtype=np.int32)
    B, width = table.shape
    old, new = [int(x) for x in old], [int(x) for x in new]
    none = (np.zeros(B + 1, np.int32), np.full(rows, -1, np.int64), np.full(rows, -1, np.int32), count)
    need = [-(-n // page) for n in new]
    held = [-(-o // page) for o in old]
    bad = any(o < 0 or n < 0 for o, n in zip(old, new)) or any(max(a, b) > width for a, b in zip(need, held))
    bad = bad or not 0 <= count <= len(stack) or sum(max(0, n - o) for o, n in zip(old, new)) > rows
    if bad or count + sum(held) - sum(need) > len(stack):
        return (*none, -1, table, stack)
    lacks = sum(need) - sum(held) - count
    if lacks > 0:
        return (*none, lacks, table, stack)
    free = [int(x) for x in stack[:count]]
    for b in range(B):
        free.extend(int(x) for x in table[b, need[b]:held[b]])
    cu, slots, positions = [0], [], []
    for b in range(B):
        for i in range(held[b], need[b]):
            table[b, i] = free.pop()
        for pos in range(old[b], new[b]):
            slots.append(int(table[b, pos // page]) * page + pos % page)
            positions.append(pos)
        cu.append(len(slots))
    if len(free) > count:
        stack[count:len(free)] = free[count:]
    pad = [-1] * (rows - len(slots))
    return (np.array(cu, np.int32), np.array(slots + pad, np.int64), np.array(positions + pad, np.int32), len(free), 0,
            table, stack)


# ------------------------------------------------------------------------------- the attention

def attention(q, cache, table, cu_q, kv_lens, page, causal, window, scale):
    """float64 (out [T, Hq, D], bound [T, Hq, D]) of float64 q [T, Hq, D] (bf16 values): the exact
    attention and how far a result of the library may be from it.

    Rows of q outside every request come back NaN. The bound, in the order of the arithmetic, with
    u = 2^-24 and A = sum_j p_j |V_j| per element:
      - a score differs by at most eps = scale * ((D + 8) u sum_d |q_d K_jd| + 2^-21 max|q| sum_d |K_jd|)
        + 6 u (|s_j| + max|s|) : FP32 sums of exact products, the rounded multiplications by the scale
        and by log2 e and the subtraction of the maximum, and the query's split into two 8-bit floats,
        exact down to 2^-21 of the row's largest element;
      - so a weight is off by a factor within exp(+-2 eps) (its own score and the maximum's cancel or
        add), by 2^-23 for the exponential (twice: rescalings), and by 2^-8 for its rounding to bf16;
      - the weights' sum has the same errors, which the quotient adds: twice (2^-8 + 2 eps + 2^-21);
      - N-term FP32 sums of the products and of the weights: 2 (N + 16) u;
      - the result is rounded to bf16: 2^-8 of it."""
    T, Hq, D = q.shape
    H = cache.shape[1]
    G = Hq // H
    out, bound = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    for b in range(len(kv_lens)):
        r0, r1, L = int(cu_q[b]), int(cu_q[b + 1]), int(kv_lens[b])
        n = r1 - r0
        if n == 0:
            continue
        pos = L - n + np.arange(n)
        j = np.arange(L)
        seen = np.ones((n, L), dtype=bool)
        if causal:
            seen &= j[None] <= pos[:, None]
        if window:
            seen &= j[None] > pos[:, None] - window
        ids = np.asarray(table[b])[j // page] if L else np.zeros(0, dtype=np.int64)
        fine = (ids >= 0) & (ids < cache.shape[0])
        seen &= fine[None]
        need = seen.any(axis=0)
        k, v = np.zeros((L, H, D)), np.zeros((L, H, D))
        if need.any():
            k[need], v[need] = read(cache, ids[need].astype(np.int64) * page + j[need] % page, page, D)
        for hq in range(Hq):
            h = hq // G
            x = q[r0:r1, hq]
            if not need.any():
                out[r0:r1, hq] = bound[r0:r1, hq] = 0.0
                continue
            out[r0:r1, hq], bound[r0:r1, hq] = attend(x, k[:, h], v[:, h], seen, scale)
    return out, bound


def attend(x, k, v, seen, scale):
    """One head of one request: (out [n, D], bound [n, D]) of rows x [n, D] over k, v [L, D] with
    seen [n, L]; the bound is the one that attention() derives."""
    D, L = x.shape[1], k.shape[0]
    u = 2.0 ** -24
    s = scale * (x @ k.T)
    mag = scale * ((D + 8) * u * (np.abs(x) @ np.abs(k).T)
                   + 2.0 ** -21 * np.abs(x).max(axis=1, keepdims=True) * np.abs(k).sum(axis=1)[None])
    masked = np.where(seen, s, -np.inf)
    top = masked.max(axis=1, keepdims=True)
    some = np.isfinite(top)
    w = np.exp(np.where(seen, s - np.where(some, top, 0.0), -np.inf))
    tot = w.sum(axis=1, keepdims=True)
    p = w / np.where(tot == 0, 1.0, tot)
    eps = np.where(seen, mag + 6 * u * np.abs(s), 0.0).max(axis=1, keepdims=True)
    eps = eps + 6 * u * np.where(seen, np.abs(s), 0.0).max(axis=1, keepdims=True)
    o, A = p @ v, p @ np.abs(v)
    rel = 2 * (2.0 ** -8 + 2 * eps + 2.0 ** -21) * 1.05 + 2 * (L + 16) * u
    return o, 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * rel * A + 1e-37
