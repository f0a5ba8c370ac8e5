"""The paged MXFP4 key/value cache and its attention: the cases that are measured, the
operators in plain form (elementary torch operations in 32 bits), and the library's calls.

The cache is one uint8 buffer of [num_pages, Hkv, page_size * D * 17 / 16] bytes. A page
holds page_size tokens (a multiple of 16) of every head; one head's block in it is, with
n = page_size / 16 tiles of 16 tokens and m = D / 32 scale blocks per token:

    K codes   [n][m][16 tokens][16 bytes]     32 E2M1 codes each, even element in the low nibble
    V codes   [n][4][16 bytes][m][4 tokens]   byte b of scale block j of token 4 g + i at [g][b][j][i]
    K scales  [n][m][16 tokens]               E8M0 bytes
    V scales  [n][16 tokens][m]

Slot s is token s % page_size of page s / page_size.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step of a serving loop: every request grows by a token, some have ended
        _tables("tables-decode", B=96, page=16, held=8192, fresh=1, ended=8, mix=1),
        # admission of a burst of prompts: many pages and many slots at once
        _tables("tables-prompts", B=48, page=64, held=0, fresh=16001, ended=0, mix=2),
        # a decoding step's new keys and values, columns of one fused projection's rows
        _write("write-decode", T=96, Hkv=8, D=128, page=16, fused=True),
        # a long prompt's keys and values, an odd number of rows
        _write("write-prompt", T=16411, Hkv=8, D=128, page=64, fused=True),
        # a single short conversation: the call whose latency is felt
        _attend("attend-one", B=1, Hkv=8, G=4, D=128, page=16, q=1, kv=1037, ragged=False, mix=3),
        # an ordinary decoding batch of ragged lengths, one place of it empty
        _attend("attend-batch", B=64, Hkv=8, G=8, D=128, page=16, q=1, kv=8192, ragged=True, empty=True, mix=4),
        # two very long contexts with few shared heads: the length is split
        _attend("attend-long", B=2, Hkv=4, G=8, D=128, page=64, q=1, kv=131072, ragged=False, mix=5),
        # drafts of four tokens checked at once, a head of its own for each query head, sliding window
        _attend("attend-draft", B=32, Hkv=12, G=1, D=64, page=32, q=4, kv=4001, ragged=True, window=1024, mix=6),
        # one whole prompt
        _attend("attend-prompt", B=1, Hkv=8, G=4, D=128, page=64, q=8192, kv=8192, ragged=False, mix=7),
        # chunks of several prompts over what they hold already, ragged on both sides
        _attend("attend-chunks", B=6, Hkv=2, G=8, D=128, page=32, q=1500, kv=12001, ragged=True, mix=8),
        # wide heads, a window that begins inside pages
        _attend("attend-wide", B=3, Hkv=2, G=5, D=256, page=16, q=2049, kv=4099, ragged=True, window=1000, mix=9),
        # decoding rows and prompt chunks in one call
        _attend("attend-mixed", B=20, Hkv=4, G=8, D=128, page=16, q=512, kv=4096, ragged=True, mostly_one=True, mix=10),
    ]


def _tables(name, **kw):
    return {"name": name, "kind": "tables", **kw}


def _write(name, **kw):
    return {"name": name, "kind": "write", **kw}


def _attend(name, **kw):
    return {"name": name, "kind": "attend", "window": 0, "causal": True, "mostly_one": False, "empty": False, **kw}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tables", "write", "attend", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 32, 64, 128])
    if kind == "tables":
        B = _log(rng, 1, 512)
        if rng.random() < 0.5:  # decoding and drafts
            return _drop(_tables("", B=B, page=page, held=_log(rng, 1, 32768), fresh=rng.randint(1, 8), ended=B // rng.randint(2, 16), mix=mix))
        fresh = max(1, min(_log(rng, 16, 32768), 500000 // B))
        return _drop(_tables("", B=B, page=page, held=rng.choice([0, _log(rng, 1, 8192)]), fresh=fresh, ended=B // rng.randint(3, 64), mix=mix))
    D = rng.choice([64, 128, 128, 256])
    if kind == "write":
        return _drop(_write("", T=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 3, 4, 8]), D=D, page=page, fused=rng.random() < 0.7))
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    shape = rng.choice(["decode", "decode", "draft", "chunk", "prompt", "mixed"])
    if shape in ("decode", "draft"):
        B = _log(rng, 1, 64)
        q = 1 if shape == "decode" else rng.randint(2, 8)
        most = (64 * 8192 * 8 * 128) // (B * Hkv * D)  # of the plain form's 32-bit keys
        kv = _log(rng, max(16, q), max(16, min(131072, most)))
    else:
        B = 1 if shape == "prompt" else _log(rng, 1, 16)
        q = _log(rng, 16, 8192 if shape == "prompt" else 2048)
        kv = q if shape == "prompt" else q + _log(rng, 1, 16384)
        # pairs as the plain form counts them, at most half of the largest listed case's
        kv = max(16, min(kv, int(16 * 8192 * 8192 * 128 / (B * Hkv * G * q * D))))
        q = min(q, kv)
    window = rng.choice([0, 0, 0, _log(rng, 64, 4096)])
    causal = window > 0 or rng.random() < 0.85
    return _drop(_attend("", B=B, Hkv=Hkv, G=G, D=D, page=page, q=q, kv=kv, ragged=B > 1 and rng.random() < 0.8, window=window,
                         causal=causal, mostly_one=shape == "mixed", empty=B > 1 and rng.random() < 0.2, mix=mix))


def _drop(case):
    del case["name"]
    return case


def _lens(case):
    """The requests' lengths of a case, on the host as a scheduler has them."""
    r = random.Random(case["mix"])
    B = case["B"]
    if case["kind"] == "tables":
        old = [r.randint(max(1, case["held"] // 8), case["held"]) if case["held"] else 0 for _ in range(B)]
        top = case["fresh"]
        new = [o + (r.randint(max(1, top // 8), top) if top > 8 else top) for o in old]
        for b in r.sample(range(B), case["ended"]):
            new[b] = 0
        return old, new
    if case["ragged"]:
        kv = [r.randint(max(1, case["kv"] // 8), case["kv"]) for _ in range(B)]
        kv[r.randrange(B)] = case["kv"]
    else:
        kv = [case["kv"]] * B
    if case["q"] <= 8:
        q = [case["q"]] * B
    elif case["mostly_one"]:
        q = [case["q"] if b % 8 == 3 or B <= 3 else 1 for b in range(B)]
    elif case["ragged"]:
        q = [r.randint(max(1, case["q"] // 8), case["q"]) for _ in range(B)]
    else:
        q = [case["q"]] * B
    q = [min(a, b) for a, b in zip(q, kv)]
    if case["empty"]:  # a padded place of the batch: rows that see nothing
        kv[0] = 0
    return q, kv


# ------------------------------------------------------------------------------- the inputs

def _quantize(x):
    """float32 [..., D] -> (E2M1 codes uint8 [..., D], E8M0 bytes uint8 [..., D / 32])."""
    y = x.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True).view(torch.int32) >> 23
    s = (top - 2).clamp_min(0)
    y = torch.ldexp(y, 127 - s)  # exact: a power of two
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_max(6.0)  # ties to even, which is the even code on each stretch
    code = torch.where(a <= 2, 2 * a, torch.where(a <= 4, a + 2, 7.0))
    code = code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    return code.flatten(-2), s.squeeze(-1).to(torch.uint8)


def _blocks(cache, n_heads, D, page):
    """Views of the four regions of every (page, head) block of a cache."""
    n, m = page // 16, D // 32
    blk = cache.view(-1, n_heads, page * D * 17 // 16)
    a, b, c = page * D // 2, page * D, page * D + page * m
    return (blk[..., :a].unflatten(-1, (n, m, 16, 16)), blk[..., a:b].unflatten(-1, (n, 4, 16, m, 4)),
            blk[..., b:c].unflatten(-1, (n, m, 16)), blk[..., c:].unflatten(-1, (n, 16, m)))


def _fill(cache, first, k, v, page):
    """Quantizes k, v [pages, heads, page, D] into the cache's pages from `first` on (inputs only)."""
    heads, D = k.shape[1], k.shape[3]
    kc, vc, ks, vs = _blocks(cache.view(-1)[first * heads * page * D * 17 // 16:][:k.shape[0] * heads * page * D * 17 // 16], heads, D, page)
    c, s = _quantize(k)
    c = c[..., 0::2] | (c[..., 1::2] << 4)
    kc.copy_(c.unflatten(-1, (-1, 16)).unflatten(2, (-1, 16)).transpose(3, 4))
    ks.copy_(s.unflatten(2, (-1, 16)).transpose(3, 4))
    c, s = _quantize(v)
    c = c[..., 0::2] | (c[..., 1::2] << 4)
    vc.copy_(c.unflatten(-1, (-1, 16)).unflatten(2, (-1, 4, 4)).permute(0, 1, 2, 3, 6, 5, 4))
    vs.copy_(s.unflatten(2, (-1, 16)))


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["kind"] == "tables":
        old, new = _lens(case)
        P = case["page"]
        held = [-(-o // P) for o in old]
        width = max([-(-n // P) for n in new] + held + [1]) + 3
        wanted = sum(max(0, -(-n // P) - h) for n, h in zip(new, held))
        total = sum(held) + wanted + 7
        ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        table = torch.randint(0, total, (case["B"], width), generator=gen, device="cuda", dtype=torch.int32)
        at = torch.arange(width, device="cuda")
        mine = at[None] < i32(held)[:, None]
        table[mine] = ids[:sum(held)]  # which pages are whose, and what an earlier step left behind
        stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        stack[:total - sum(held)] = ids[sum(held):]
        tokens = sum(max(0, n - o) for o, n in zip(old, new))
        return {"kind": "tables", "old": i32(old), "new": i32(new), "table": table, "stack": stack, "count": i32([total - sum(held)]),
                "page": P, "rows": tokens + 5}  # rows: a padded batch's
    D, Hkv, P = case["D"], case["Hkv"], case["page"]
    if case["kind"] == "write":
        T = case["T"]
        pages = -(-T // P) + 3
        if case["fused"]:  # columns of the rows that one projection wrote: 2 Hkv query heads, then keys, then values
            rows = _normal(gen, T, 4 * Hkv, D)
            rows[..., 2 * Hkv:, : D // 16] *= 8.0  # keys and values have channels that stand out
            rows = rows.to(torch.bfloat16)
            k, v = rows[:, 2 * Hkv:3 * Hkv], rows[:, 3 * Hkv:]
        else:
            k, v = _normal(gen, T, Hkv, D).to(torch.bfloat16), _normal(gen, T, Hkv, D).to(torch.bfloat16)
        perm = torch.randperm(pages, generator=gen, device="cuda")
        if T <= 512:  # a token of each request, anywhere
            slots = torch.randperm(pages * P, generator=gen, device="cuda")[:T]
        else:  # a prompt's: whole pages, in order inside each
            pos = torch.arange(T, device="cuda") + P // 3
            slots = perm[pos // P] * P + pos % P
        cache = torch.randint(0, 256, (pages, Hkv, P * D * 17 // 16), generator=gen, device="cuda", dtype=torch.uint8)
        return {"kind": "write", "k": k, "v": v, "slots": slots.to(torch.int64), "cache": cache, "page": P, "Hkv": Hkv, "D": D}
    q_lens, kv_lens = _lens(case)
    B, Hq, T = case["B"], Hkv * case["G"], sum(q_lens)
    each = [-(-n // P) for n in kv_lens]
    width, used = max(each) + 2, sum(each)
    pages = used + 5
    cache = torch.empty((pages, Hkv, P * D * 17 // 16), dtype=torch.uint8, device="cuda")
    part = max(1, (1 << 28) // (Hkv * P * D * 4))
    tilt = torch.ones(D, device="cuda")
    tilt[: D // 32] = 4.0  # key channels that stand out
    for first in range(0, pages, part):
        n = min(part, pages - first)
        _fill(cache, first, _normal(gen, n, Hkv, P, D) * tilt, _normal(gen, n, Hkv, P, D), P)
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    mine = torch.arange(width, device="cuda")[None] < i32(each)[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[mine] = ids[:used]
    # past a request's end its last page holds bytes that were never written: the scales' NaN pattern among them
    _, _, ks, vs = _blocks(cache, Hkv, D, P)
    some = [b for b in range(B) if kv_lens[b]]
    last = table[some, [each[b] - 1 for b in some]].long()
    left = i32([kv_lens[b] - (each[b] - 1) * P for b in some])
    tail = (torch.arange(P, device="cuda")[None] >= left[:, None]).view(-1, 1, P // 16, 1, 16)
    ks[last] = torch.where(tail, 255, ks[last]).to(torch.uint8)
    vs[last] = torch.where(tail.transpose(3, 4), 255, vs[last]).to(torch.uint8)
    rows = _normal(gen, T, Hq + 2 * Hkv, D).to(torch.bfloat16)
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    return {"kind": "attend", "q": rows[:, :Hq] * 2, "cache": cache, "table": table, "cu_q": i32(starts), "kv_lens": i32(kv_lens),
            "page": P, "Hkv": Hkv, "D": D, "causal": case["causal"], "window": case["window"], "scale": D ** -0.5,
            "max_q": max(q_lens), "max_kv": max(kv_lens)}


# ------------------------------------------------------------------------------- one pass

def run(state):
    return {"tables": _run_tables, "write": _run_write, "attend": _run_attend}[state["kind"]](state)


def _run_tables(s):
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        cu_q, slots, positions, count, status = mx.mx_kv_tables(s["old"], s["new"], s["table"], s["stack"], s["count"], s["page"], s["rows"])
        return {"cu_q": cu_q, "slots": slots, "positions": positions, "count": count, "status": status, "table": s["table"], "stack": s["stack"]}
    return _plain_tables(s["old"], s["new"], s["table"], s["stack"], s["count"], s["page"], s["rows"])


def _run_write(s):
    """The write, and the written rows as the cache stands for them."""
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        mx.mx_kv_write(s["k"], s["v"], s["slots"], s["cache"], s["page"])
        k, v = mx.mx_kv_read(s["cache"], s["slots"], s["Hkv"], s["D"], s["page"])
        return {"k": k, "v": v}
    _plain_write(s["k"], s["v"], s["slots"], s["cache"], s["page"])
    k, v = _plain_read(s["cache"], s["slots"], s["Hkv"], s["D"], s["page"])
    return {"k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _run_attend(s):
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        return mx.mx_kv_attention(s["q"], s["cache"], s["table"], s["cu_q"], s["kv_lens"], s["Hkv"], s["page"], causal=s["causal"],
                                  window=s["window"], scale=s["scale"], max_q=s["max_q"], max_kv=s["max_kv"])
    return _plain_attend(s)


def _plain_tables(old, new, table, stack, count, page, rows):
    B, width = table.shape
    old, new = old.long(), new.long()
    held, want = (old + page - 1) // page, (new + page - 1) // page
    zero = torch.zeros(1, dtype=torch.int64, device=old.device)
    cu = torch.cat([zero, torch.cumsum((new - old).clamp_min(0), 0)])
    cu_out = torch.cat([zero, torch.cumsum((held - want).clamp_min(0), 0)])  # pages given back
    cu_in = torch.cat([zero, torch.cumsum((want - held).clamp_min(0), 0)])   # pages taken
    have = count.long()
    short = cu_in[-1:] - cu_out[-1:] - have
    ok = short <= 0
    # the stack with what is given back on top, in the requests' order
    at = torch.arange(stack.numel(), device=old.device)
    k = at - have
    b = torch.searchsorted(cu_out[1:], k, right=True).clamp(0, B - 1)
    back = table[b, (want[b] + k - cu_out[b]).clamp(0, width - 1)]
    full = torch.where((k >= 0) & (k < cu_out[-1]), back, stack)
    left = have + cu_out[-1] - cu_in[-1]
    # the new rows
    t = torch.arange(rows, device=old.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(B - 1)
    live = (t < cu[-1]) & ok
    pos = old[b] + t - cu[b]
    blk = (pos // page).clamp(0, width - 1)
    taken = have + cu_out[-1] - 1 - (cu_in[b] + blk - held[b])
    fresh = full[taken.clamp(0, stack.numel() - 1)]
    id_ = torch.where(blk < held[b], table[b, blk], fresh)
    slots = torch.where(live, id_.long() * page + pos % page, -1)
    positions = torch.where(live, pos, -1).int()
    # the grown requests' new entries
    col = torch.arange(width, device=old.device)[None]
    grows = (col >= held[:, None]) & (col < want[:, None]) & ok
    taken = have + cu_out[-1] - 1 - (cu_in[:-1, None] + col - held[:, None])
    new_table = torch.where(grows, full[taken.clamp(0, stack.numel() - 1)], table)
    new_stack = torch.where(ok & (at >= have) & (at < left), full, stack)
    return {"cu_q": torch.where(ok, cu, 0).int(), "slots": slots, "positions": positions, "count": torch.where(ok, left, have).int(),
            "status": short.clamp_min(0).int(), "table": new_table, "stack": new_stack}


def _plain_write(k, v, slots, cache, page):
    heads, D = k.shape[1:]
    kc, vc, ks, vs = _blocks(cache, heads, D, page)
    p, t = slots // page, slots % page
    n, r = t // 16, t % 16
    c, s = _quantize(k.float())
    kc[p, :, n, :, r] = (c[..., 0::2] | (c[..., 1::2] << 4)).unflatten(-1, (-1, 16))
    ks[p, :, n, :, r] = s
    c, s = _quantize(v.float())
    vc[p, :, n, r // 4, :, :, r % 4] = (c[..., 0::2] | (c[..., 1::2] << 4)).unflatten(-1, (-1, 16)).transpose(2, 3)
    vs[p, :, n, r] = s


def _values(codes, scales):
    """float32 [..., D] of packed codes [..., m, 16] and scale bytes [..., m]."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return torch.ldexp(x, scales.int().unsqueeze(-1) - 127).flatten(-2)


def _plain_read(cache, slots, heads, D, page):
    kc, vc, ks, vs = _blocks(cache, heads, D, page)
    p, t = slots // page, slots % page
    n, r = t // 16, t % 16
    return (_values(kc[p, :, n, :, r], ks[p, :, n, :, r]),
            _values(vc[p, :, n, r // 4, :, :, r % 4].transpose(2, 3), vs[p, :, n, r]))


def _plain_attend(s):
    q, page, D, Hkv = s["q"], s["page"], s["D"], s["Hkv"]
    T, Hq = q.shape[:2]
    B, G = s["kv_lens"].numel(), Hq // Hkv
    width = -(-s["max_kv"] // page)
    # the requests' pages, gathered and decoded: [B, Hkv, width * page, D]
    kc, vc, ks, vs = _blocks(s["cache"][s["table"][:, :width].clamp_min(0).long()].flatten(0, 1), Hkv, D, page)
    k = _values(kc.transpose(3, 4), ks.transpose(3, 4)).unflatten(0, (B, width)).transpose(1, 2).reshape(B, Hkv, width * page, D)
    v = _values(vc.permute(0, 1, 2, 3, 6, 5, 4).flatten(3, 4), vs).unflatten(0, (B, width)).transpose(1, 2).reshape(B, Hkv, width * page, D)
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=q.device)
    rows = (cu[:-1, None] + i).clamp_max(T - 1)
    x = q[rows].float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * s["max_q"], D)
    j = torch.arange(width * page, device=q.device)
    pos = (kv - n)[:, None] + i  # [B, max_q]
    seen = (j[None, None] < kv[:, None, None]) & (pos >= 0)[..., None] if s["causal"] else (j < kv[:, None, None]).expand(B, s["max_q"], -1)
    if s["causal"]:
        seen = seen & (j <= pos[..., None])
    if s["window"]:
        seen = seen & (j > pos[..., None] - s["window"])
    v = torch.where((j < kv[:, None])[:, None, :, None], v, 0.0)  # what was never written is not read
    p = torch.matmul(x, k.transpose(2, 3)).unflatten(2, (G, -1)).mul_(s["scale"])
    p = p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (G, -1)) / torch.where(total == 0, 1.0, total)
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(B - 1)
    return o.permute(0, 3, 1, 2, 4)[b, t - cu[b]].flatten(1, 2).to(torch.bfloat16)


# ------------------------------------------------------------------------------- what a pass needs

def work(case):
    if case["kind"] == "tables":
        old, new = _lens(case)
        P = case["page"]
        moved = sum(abs(-(-n // P) - -(-o // P)) for o, n in zip(old, new))
        tokens = sum(max(0, n - o) for o, n in zip(old, new))
        return {"bytes": 12 * len(old) + 8 * moved + 12 * tokens + 16, "flops": 0}
    D, Hkv = case["D"], case["Hkv"]
    if case["kind"] == "write":  # rows in, cache out; cache in, rows out
        return {"bytes": case["T"] * (2 * Hkv * D * 2 * 2 + 2 * Hkv * D * 17 // 16 + 16), "flops": 0}
    q_lens, kv_lens = _lens(case)
    pairs, tokens = 0, 0
    for n, kv in zip(q_lens, kv_lens):
        n = min(n, kv) if case["causal"] else n  # queries before the first key see nothing
        first = kv - n  # the first query's position
        w = case["window"] or kv + 1
        if case["causal"]:
            full = max(0, min(n, w - 1 - first))  # queries whose window reaches the beginning
            pairs += full * (first + 1) + full * (full - 1) // 2 + (n - full) * w
            tokens += min(kv, n + w - 1)
        else:
            pairs += n * kv
            tokens += kv
    Hq = Hkv * case["G"]
    return {"bytes": 4 * sum(q_lens) * Hq * D + tokens * Hkv * D * 17 // 16 + 4 * tokens // case["page"], "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "tables":
        return _exact_tables(s)
    if case["kind"] == "write":
        return {"k": _exact_mx(s["k"]), "v": _exact_mx(s["v"])}
    q, G, page, D = s["q"].double(), case["G"], s["page"], s["D"]
    kc, vc, ks, vs = _blocks(s["cache"], s["Hkv"], D, page)
    cu, kv = s["cu_q"].tolist(), s["kv_lens"].tolist()
    if work(case)["flops"] > 3e12 or sum(kv) * s["Hkv"] * D > 2e9:
        return None
    out = torch.zeros_like(q)
    for b, L in enumerate(kv):
        n = cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-L // page)].long()
        # bytes of one token in a row: [tokens, heads, D / 2]
        kb = kc[ids].permute(0, 2, 4, 1, 3, 5).reshape(-1, s["Hkv"], D // 2)[:L]
        vb = vc[ids].permute(0, 2, 3, 6, 1, 5, 4).reshape(-1, s["Hkv"], D // 2)[:L]
        ke = ks[ids].permute(0, 2, 4, 1, 3).reshape(-1, s["Hkv"], D // 32)[:L]
        ve = vs[ids].permute(0, 2, 3, 1, 4).reshape(-1, s["Hkv"], D // 32)[:L]
        for h in range(s["Hkv"]):
            kh, vh = _exact_decode(kb[:, h], ke[:, h]), _exact_decode(vb[:, h], ve[:, h])
            for g in range(h * G, h * G + G):
                for i in range(0, n, 2048):
                    at = torch.arange(i, min(n, i + 2048), device=q.device)[:, None] + (L - n)
                    j = torch.arange(L, device=q.device)[None]
                    hide = torch.zeros((at.numel(), L), dtype=torch.bool, device=q.device)
                    if s["causal"]:
                        hide |= j > at
                    if s["window"]:
                        hide |= j <= at - s["window"]
                    z = (q[cu[b] + i:cu[b] + i + at.numel(), g] @ kh.T) * s["scale"]
                    z[hide] = -math.inf
                    z = torch.softmax(z, -1)
                    out[cu[b] + i:cu[b] + i + at.numel(), g] = torch.nan_to_num(z, nan=0.0) @ vh
    return out


def _exact_decode(packed, scales):
    """float64 [L, D] of bytes [L, D / 2] and scale bytes [L, D / 32], from the format's bits."""
    nib = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).double()
    sign = 1 - 2 * torch.floor(nib / 8)
    nib = nib % 8
    e, m = torch.floor(nib / 2), nib % 2
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    return sign * mag * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _exact_mx(x):
    """The nearest E2M1 value, ties to the even code, at the block's power of two; in 64 bits."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top == 0, torch.ones_like(top), top)))
    e = torch.where(top == 0, torch.full_like(e, -127), (e - 2).clamp_min(-127))
    y = x.abs() / torch.exp2(e)
    values = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    near = torch.zeros_like(y)
    for lo in range(7):
        mid = (values[lo] + values[lo + 1]) / 2
        near = torch.where((y > mid) | ((y == mid) & (lo % 2 == 1)), values[lo + 1], near)
    return (torch.sign(x) * near * torch.exp2(e)).flatten(-2)


def _exact_tables(s):
    """The same by a stack and loops on the host."""
    old, new, page = s["old"].tolist(), s["new"].tolist(), s["page"]
    table, stack, count = s["table"].tolist(), s["stack"].tolist(), int(s["count"])
    free = stack[:count]
    for b, (o, n) in enumerate(zip(old, new)):
        free += table[b][-(-n // page):-(-o // page)]
    slots, positions, cu = [], [], [0]
    for b, (o, n) in enumerate(zip(old, new)):
        for blk in range(-(-o // page), -(-n // page)):
            table[b][blk] = free.pop()
        slots += [table[b][p // page] * page + p % page for p in range(o, n)]
        positions += range(o, n)
        cu.append(len(slots))
    pad = [-1] * (s["rows"] - len(slots))
    stack[count:] = (free[count:] + stack[max(count, len(free)):])[:len(stack) - count]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"cu_q": i32(cu), "slots": torch.tensor(slots + pad), "positions": i32(positions + pad), "count": i32([len(free)]),
            "status": i32([0]), "table": i32(table), "stack": i32(stack)}
