"""CPU oracle for routing to experts, its sorted tables, the cache's append and the verification
of drafts.

TEST INFRASTRUCTURE ONLY. The test suite is the only caller; the product library never
imports, links or runs anything here. Everything is NumPy in float64 or integers, written
from the definitions in include/mx.h.
"""
from __future__ import annotations

import math

import numpy as np

from . import mx_act_oracle as A
from . import mx_kv_oracle as KV

FLT_MAX = float(np.finfo(np.float32).max)
BF16_MAX = 2.0 ** 128 - 2.0 ** 120


# ------------------------------------------------------------------------------- routing

def truncated(x: np.ndarray) -> np.ndarray:
    """float64 values as they are compared: the low 10 mantissa bits off, -0 as 0."""
    x = np.clip(np.asarray(x, dtype=np.float64) + 0.0, -1e300, 1e300)
    return (x.view(np.uint64) & ~np.uint64(1023)).view(np.float64)


def rounded(x: float) -> float:
    """A group's value as it is compared: rounded to those bits, halves away from 0."""
    x = np.clip(np.array([x], dtype=np.float64), -1e300, 1e300)
    return float(truncated((x.view(np.uint64) + np.uint64(512)).view(np.float64))[0])


def route(logits, topk, bias=None, sigmoid=False, groups=1, topk_groups=1, group_top=2, renormalize=True, scale=1.0, rows=None,
          largest=FLT_MAX):
    """(ids int32 [T, topk], weights float64 [T, topk]) token by token; logits are float32 values of a type
    whose largest number is `largest`."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    ids, weights = np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    for t in range(T if rows is None else max(0, min(T, rows))):
        l = np.minimum(logits[t], largest)
        ok = l > -math.inf
        if bias is not None:
            with np.errstate(invalid="ignore"):
                b = np.minimum(np.asarray(bias, dtype=np.float64), FLT_MAX)
                ok &= b > -math.inf
        if not ok.any():
            continue
        with np.errstate(all="ignore"):
            if sigmoid:
                s = np.where(ok, 1 / (1 + np.exp(-l)), 0.0)
            else:
                s = np.where(ok, np.exp(l - l[ok].max()), 0.0)
                s = s / s.sum()
            full = l if bias is None else s + b
            c = truncated(full)
            by = s if bias is None and group_top == 2 else full
        left = [e for e in range(E) if ok[e]]
        if groups > 1:
            n = E // groups
            value = {}
            for g in range(groups):
                best = sorted((by[e] for e in range(g * n, g * n + n) if ok[e]), reverse=True)[:group_top]
                if best:
                    value[g] = rounded(best[0] + best[1] if len(best) > 1 else best[0])
            keep = sorted(value, key=lambda g: (-value[g], g))[:topk_groups]
            left = [e for e in left if e // n in keep]
        chosen = sorted(left, key=lambda e: (-c[e], e))[:topk]
        w = s[chosen]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(chosen)], weights[t, :len(chosen)] = chosen, scale * w
    return ids, weights


def sort(ids, E, first=0):
    """(expert_offsets, row_token, token_rows), expert by expert."""
    ids = np.asarray(ids)
    T, topk = ids.shape
    flat = ids.reshape(-1).astype(np.int64) - first
    offsets, row_token, rows = [0], np.full(T * topk, -1, np.int32), np.full(T * topk, -1, np.int32)
    for e in range(E):
        at = np.flatnonzero(flat == e)
        row_token[offsets[-1]:offsets[-1] + at.size] = at // topk
        rows[at] = offsets[-1] + np.arange(at.size)
        offsets.append(offsets[-1] + at.size)
    return np.array(offsets, np.int32), row_token, rows.reshape(T, topk)


# ------------------------------------------------------------------------------- append

def norm_rotate(x, positions, weight, eps, inv_freq, pairs, rope_scale=1.0):
    """(y, size) float64 [T, H, D] of float64 x: the normed and rotated heads, and the sum of the
    magnitudes of the one or two terms that each element of y is made of."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        mean = (x * x).mean(axis=-1, keepdims=True) + np.float64(np.float32(eps))
        x = x / np.sqrt(np.maximum(mean, 2.0 ** -126)) * np.asarray(weight, dtype=np.float64)
    y, size = x.copy(), np.abs(x)
    if inv_freq is not None and len(inv_freq):
        n = len(inv_freq)
        angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None]
        c, s = np.cos(angle)[:, None] * rope_scale, np.sin(angle)[:, None] * rope_scale
        ia = np.arange(n) * 2 if pairs else np.arange(n)
        ib = ia + 1 if pairs else ia + n
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia], size[..., ib] = np.abs(a * c) + np.abs(b * s), np.abs(a * s) + np.abs(b * c)
    return y, size


def query_bound(y, size):
    """How far a query may be: in FP32, with u = 2^-24, each of its two terms by its coefficient, cosine
    or sine (2 u) times rope_scale and weight (2 u), and by its product (u, one of the two); their sum
    (u); the norm's factor: the sum of squares, 8 fused products in a lane and up to 5 sums over lanes,
    all of one sign, 13 u, of which the root takes half; the mean and eps in one fused product (u, half),
    the root itself (2 u); the product with it (u). In all 6 + 7 + 2 + 1 = 16 u of the terms' magnitudes,
    20 allowed for the second order and 1 / D; then half a step of bf16, 2^-8 of the value (2^-134 among
    its subnormals)."""
    return (2.0 ** -8 * np.abs(y) + 20 * 2.0 ** -24 * size) * (1 + 2.0 ** -8) + 2.0 ** -133


def append(cache, k, v_bits, positions, slots, page, weight, eps, inv_freq, pairs, rope_scale=1.0):
    """Keys (float64 values [T, H, D]) normed, rotated, rounded to float32 and, with v (bf16 bits), into
    cache uint8 [pages, H, block]; rows of a position below 0 or a slot outside are skipped."""
    T, H, D = k.shape
    y, _ = norm_rotate(k, positions, weight, eps, inv_freq, pairs, rope_scale)
    y = y.astype(np.float32).astype(np.float64)
    inside = np.where(np.asarray(positions) < 0, -1, slots)
    KV.write(cache, np.zeros((T, H, D), np.uint16), v_bits, inside, page)
    mk, _, mks, _ = KV._maps(page, D)
    q, s = A.quantize_mx_values(y.reshape(T * H, D))
    q, s = q.reshape(T, H, D // 32, 16), s.reshape(T, H, D // 32)
    for t, slot in enumerate(inside):
        if 0 <= slot < cache.shape[0] * page:
            p, tok = divmod(int(slot), page)
            for h in range(H):
                cache[p, h, mk[tok]] = q[t, h]
                cache[p, h, mks[tok]] = s[t, h]


# ------------------------------------------------------------------------------- verification

def verify(p, q, tokens, cu_q, kv_lens, accept, sample):
    """(out_tokens, accepted, new_lens) request by request; q may be None."""
    T, V = p.shape
    clean = lambda x: np.where(x > 0, x, 0).astype(np.float64)  # noqa: E731  (NaN is not > 0)
    out, accepted, lens = np.full(T, -1, np.int32), [], []
    for b, kv in enumerate(kv_lens):
        r0 = min(max(int(cu_q[b]), 0), T)
        n = min(max(int(cu_q[b + 1]), r0), T) - r0
        acc = 0
        while acc < n - 1:
            x = int(tokens[r0 + acc + 1])
            if not 0 <= x < V:
                break
            px, qx = clean(p[r0 + acc, x]), 1.0 if q is None else clean(q[r0 + acc, x])
            if not float(accept[r0 + acc]) * float(qx) < float(px):
                break
            out[r0 + acc] = x
            acc += 1
        if n > 0:
            w = whole = clean(p[r0 + acc])
            if acc < n - 1:
                x = int(tokens[r0 + acc + 1])
                if q is not None:
                    w = np.maximum(whole - clean(q[r0 + acc]), 0)
                elif 0 <= x < V:
                    w = whole.copy()
                    w[x] = 0
                if not w.sum() > 0:
                    w = whole
            if w.sum() > 0:
                run = np.cumsum(w)
                u = float(sample[b])
                goal = (min(u, 1.0) if u > 0 else 0.0) * run[-1]  # NaN counts as 0
                past = np.flatnonzero((run > goal) & (w > 0))
                out[r0 + acc] = past[0] if past.size else np.flatnonzero(w > 0)[-1]
        accepted.append(acc)
        lens.append(int(kv) - (max(n, 1) - 1 - acc))
    return out, np.array(accepted, np.int32), np.array(lens, np.int32)
