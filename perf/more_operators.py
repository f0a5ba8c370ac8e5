"""Expert routing and its sorted tables, appending to the paged MXFP4 cache, and the
verification of drafts: the cases that are measured, the operators in plain form (elementary
torch operations), and the library's calls.

The cache's layout is that of include/mx.h: one uint8 buffer of [num_pages, heads,
page_size * D * 17 / 16] bytes; with n = page_size / 16 and m = D / 32 a block holds

    K codes   [n][m][16 tokens][16 bytes]     32 E2M1 codes each, even element in the low nibble
    V codes   [n][4][16 bytes][m][4 tokens]   byte b of scale block j of token 4 g + i at [g][b][j][i]
    K scales  [n][m][16 tokens]               E8M0 bytes
    V scales  [n][16 tokens][m]
"""
import math
import random

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decoding step's few tokens over very many experts: the call whose latency is felt
        _route("route-step", T=16, E=896, topk=16),
        # a chunk of a prompt, sigmoid scores with a bias for balance, experts in groups, FP32 logits
        _route("route-groups", T=4099, E=256, topk=8, score="sigmoid", bias=True, groups=8, topk_groups=4, scale=2.5, fp32=True),
        # a long prompt, an odd number of tokens, the last of them padding
        _route("route-prompt", T=16411, E=896, topk=16, padded=27),
        # a decoding step's choices into tables
        _sort("sort-step", T=16, E=896, topk=16),
        # a prompt's
        _sort("sort-chunk", T=4096, E=896, topk=16),
        # many prompts', for the half of the experts that one of several devices holds
        _sort("sort-share", T=65537, E=256, topk=8, first=64, local=128),
        # a decoding step of a padded batch at far positions: norms, rotation, columns of one fused projection
        _append("append-step", T=101, padded=5, Hkv=8, G=4, D=128, page=16, norms=True, far=131071),
        # a prompt's chunk, a head of its own for each query head, part of each head rotated in neighbouring pairs
        _append("append-chunk", T=2051, Hkv=12, G=1, D=64, page=32, rope="pairs", rot=32, far=9001),
        # one long prompt
        _append("append-prompt", T=16411, Hkv=8, G=4, D=128, page=64, norms=True, far=0),
        # one request's five drafts against a sampled draft's probabilities
        _verify("verify-one", B=1, most=6, V=131072, ragged=False, mix=1),
        # an ordinary batch, ragged drafts
        _verify("verify-batch", B=64, most=5, V=131072, mix=2),
        # drafts without probabilities of their own (looked up in the text), rows of an odd length
        _verify("verify-lookup", B=150, most=4, V=50021, sampled=False, mix=3),
    ]


def _route(name, **kw):
    return {"name": name, "kind": "route", "score": "softmax", "bias": False, "groups": 1, "topk_groups": 1, "group_top": 2,
            "renormalize": True, "scale": 1.0, "fp32": False, "padded": 0, **kw}


def _sort(name, **kw):
    return {"name": name, "kind": "sort", "first": 0, "local": kw["E"], **kw}


def _append(name, **kw):
    return {"name": name, "kind": "append", "padded": 0, "rope": "halves", "rot": kw["D"], "norms": False, **kw}


def _verify(name, **kw):
    return {"name": name, "kind": "verify", "ragged": True, "sampled": True, **kw}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "sort", "append", "verify"])
    if kind in ("route", "sort"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 320, 512, 896, 1000])
        topk = rng.randint(1, min(16, E // 2))
        if kind == "sort":
            share = rng.choice([1, 1, 2, 4])
            local = E // share
            return _drop(_sort("", T=_log(rng, 1, 65536 * 8 // topk), E=E, topk=topk, first=rng.randrange(share) * local, local=local))
        groups = rng.choice([1, 1] + [g for g in (2, 4, 5, 8, 16) if E % g == 0 and E // g >= 2])
        keep = rng.randint(1, groups)
        topk = min(topk, keep * (E // groups))
        T = _log(rng, 1, 16384)
        return _drop(_route("", T=T, E=E, topk=topk, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                            topk_groups=keep, group_top=rng.choice([1, 2]), renormalize=rng.random() < 0.6,
                            scale=rng.choice([1.0, 2.5, 16.0]), fp32=rng.random() < 0.4, padded=T // 8 if rng.random() < 0.3 else 0))
    if kind == "append":
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8])
        T = _log(rng, 1, max(1, min(16384, 16384 * 48 * 128 // (Hkv * (G + 2) * D))))
        return _drop(_append("", T=T, padded=T // 10 if rng.random() < 0.3 else 0, Hkv=Hkv, G=G, D=D, page=rng.choice([16, 32, 64, 128]),
                             rope=rng.choice(["halves", "pairs"]), rot=rng.choice([D, D, D // 2, D // 4, 0]), norms=rng.random() < 0.6,
                             far=rng.choice([0, _log(rng, 100, 1000000)])))
    V = _log(rng, 1000, 262144)
    most = rng.randint(1, 9)
    return _drop(_verify("", B=_log(rng, 1, max(1, min(512, 64 * 5 * 131072 // (V * most)))), most=most, V=V, ragged=rng.random() < 0.7,
                         sampled=rng.random() < 0.7, mix=rng.randrange(1 << 30)))


def _drop(case):
    del case["name"]
    return case


def _rows_of(case):
    """The rows of each request of a verify case: its last token and its drafts."""
    r = random.Random(case["mix"])
    return [r.randint(1, case["most"]) if case["ragged"] else case["most"] for _ in range(case["B"])]


# ------------------------------------------------------------------------------- the inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"route": _prepare_route, "sort": _prepare_sort, "append": _prepare_append, "verify": _prepare_verify}[case["kind"]](case, gen)
    s["kind"] = case["kind"]
    return s


def _prepare_route(case, gen):
    T, E = case["T"], case["E"]
    logits = _normal(gen, T, E) * 1.5 + _normal(gen, E) * 0.7  # some experts are asked for more than others
    s = {k: case[k] for k in ("topk", "score", "groups", "topk_groups", "group_top", "renormalize", "scale")}
    s["logits"] = logits if case["fp32"] else logits.to(torch.bfloat16)
    s["bias"] = _normal(gen, E) * 0.05 if case["bias"] else None
    s["num_rows"] = torch.tensor([T - case["padded"]], dtype=torch.int32, device="cuda") if case["padded"] else None
    return s


def _prepare_sort(case, gen):
    T, E = case["T"], case["E"]
    ids = torch.empty((T, case["topk"]), dtype=torch.int32, device="cuda")
    liked = _normal(gen, E) * 0.7
    for t in range(0, T, 16384):
        n = min(16384, T - t)
        ids[t:t + n] = torch.topk(_normal(gen, n, E) + liked, case["topk"]).indices.to(torch.int32)
    return {"ids": ids, "E": case["local"], "first": case["first"]}


def _prepare_append(case, gen):
    T, H, G, D, P = (case[k] for k in ("T", "Hkv", "G", "D", "page"))
    Hq = H * G
    rows = _normal(gen, T, Hq + 2 * H, D)
    rows[..., Hq:, :D // 16] *= 8.0  # keys and values have channels that stand out
    rows = rows.to(torch.bfloat16)  # one projection's: queries, keys, values
    pages = -(-T // P) + 3
    perm = torch.randperm(pages, generator=gen, device="cuda")
    live = T - case["padded"]
    if case["far"] and T <= 512:  # a token of each request, anywhere
        slots = torch.randperm(pages * P, generator=gen, device="cuda")[:T]
        pos = torch.randint(0, case["far"] + 1, (T,), generator=gen, device="cuda")
    else:  # a prompt's or a chunk's: whole pages, in order inside each
        at = torch.arange(T, device="cuda") + P // 3
        slots = perm[at // P] * P + at % P
        pos = torch.arange(T, device="cuda") + case["far"]
    slots[live:], pos[live:] = -1, -1
    i = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    return {"q": rows[:, :Hq], "k": rows[:, Hq:Hq + H], "v": rows[:, Hq + H:], "positions": pos.to(torch.int32),
            "slots": slots.to(torch.int64), "page": P, "rope": case["rope"],
            "cache": torch.randint(0, 256, (pages, H, P * D * 17 // 16), generator=gen, device="cuda", dtype=torch.uint8),
            "inv_freq": (500000.0 ** (-2.0 * i / max(1, case["rot"]))).to(torch.float32) if case["rot"] else None,
            "q_weight": 1 + 0.2 * _normal(gen, D) if case["norms"] else None,
            "k_weight": 1 + 0.2 * _normal(gen, D) if case["norms"] else None, "eps": 1e-6,
            # padding rows are left as they were
            "q_out": torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda"),
            "k_out": torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"),
            "v_out": torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")}


def _prepare_verify(case, gen):
    n, V = _rows_of(case), case["V"]
    T = sum(n) + 3  # a padded batch's rows
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    z = _normal(gen, T, V) * 2.5
    target = torch.softmax(z, -1)
    z += _normal(gen, T, V) * 0.7  # the draft model is nearly of the target's mind
    draft = torch.softmax(z, -1)
    if case["sampled"]:
        guess = (draft / -torch.log(_uniform(gen, T, V).clamp_min(1e-30))).argmax(-1)  # a sample of the draft's
    else:
        guess = (target * (1 + _uniform(gen, T, V))).argmax(-1)
    tokens = torch.randint(0, V, (T,), generator=gen, device="cuda")
    tokens[1:] = guess[:-1]  # row t's guess is drafted as the next row's token
    kv = torch.tensor([x + 40 for x in n], dtype=torch.int32, device="cuda") + torch.randint(0, 4000, (len(n),), generator=gen, device="cuda", dtype=torch.int32)
    return {"target": target, "draft": draft if case["sampled"] else None, "tokens": tokens.to(torch.int32),
            "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"), "kv_lens": kv, "accept": _uniform(gen, T),
            "sample": _uniform(gen, len(n)), "max_q": max(n)}


# ------------------------------------------------------------------------------- one pass

def run(state):
    return {"route": _run_route, "sort": _run_sort, "append": _run_append, "verify": _run_verify}[state["kind"]](state)


def _run_route(s):
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        score = mx.MX_SCORE_SOFTMAX if s["score"] == "softmax" else mx.MX_SCORE_SIGMOID
        ids, weights = mx.mx_moe_route(s["logits"], s["topk"], bias=s["bias"], score=score, groups=s["groups"], topk_groups=s["topk_groups"],
                                       group_top=s["group_top"], renormalize=s["renormalize"], scale=s["scale"], num_rows=s["num_rows"])
        return {"ids": ids, "weights": weights}
    return _plain_route(s)


def _run_sort(s):
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        offsets, row_token, token_rows = mx.mx_moe_sort(s["ids"], s["E"], first_expert=s["first"])
        return {"offsets": offsets, "row_token": row_token, "token_rows": token_rows}
    return _plain_sort(s["ids"], s["E"], s["first"])


def _run_append(s):
    """The append, and the written rows as the cache stands for them."""
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        rope = mx.MX_ROPE_HALVES if s["rope"] == "halves" else mx.MX_ROPE_PAIRS
        q = mx.mx_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cache"], s["page"], inv_freq=s["inv_freq"], rope=rope,
                            q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], q_out=s["q_out"])
        k, v = mx.mx_kv_read(s["cache"], s["slots"], s["k"].shape[1], s["k"].shape[2], s["page"], k_out=s["k_out"], v_out=s["v_out"])
        return {"q": q, "k": k, "v": v}
    return _plain_append(s)


def _run_verify(s):
    if own:
        import mxfp4_quantized_gemm_inline_amd as mx
        tokens, accepted, lens = mx.mx_verify_drafts(s["target"], s["draft"], s["tokens"], s["cu_q"], s["kv_lens"], s["accept"], s["sample"])
        return {"tokens": tokens, "accepted": accepted, "lens": lens}
    return _plain_verify(s)


def _plain_route(s):
    """In 64 bits: which of two scores is larger is asked next to borders."""
    x = s["logits"].double()
    T, E = x.shape
    G, k = s["groups"], s["topk"]
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    choice = x if s["bias"] is None else p + s["bias"].double()  # without a bias the logits stand in the scores' order
    if G > 1:
        value = choice if s["bias"] is not None or s["group_top"] == 1 else p
        value = value.unflatten(1, (G, E // G)).sort(dim=-1, descending=True).values[..., :s["group_top"]].sum(-1)
        best = value.sort(dim=-1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        choice = choice.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * s["scale"]
    if s["num_rows"] is not None:
        pad = (torch.arange(T, device=x.device) >= s["num_rows"])[:, None]
        ids, w = torch.where(pad, -1, ids), torch.where(pad, 0.0, w)
    return {"ids": ids.to(torch.int32), "weights": w.to(torch.float32)}


def _plain_sort(ids, E, first):
    T, k = ids.shape
    e = ids.reshape(-1).long() - first
    e = torch.where((e >= 0) & (e < E), e, E)  # others' experts behind the last
    _, order = torch.sort(e, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device).index_add_(0, e, torch.ones_like(e))
    offsets = torch.cat([counts.new_zeros(1), torch.cumsum(counts[:E], 0)])
    at = torch.arange(T * k, device=e.device)
    row_token = torch.where(at < offsets[E], order // k, -1)
    rows = torch.empty_like(order)
    rows[order] = at
    rows = torch.where(e < E, rows, -1)
    return {"offsets": offsets.to(torch.int32), "row_token": row_token.to(torch.int32), "token_rows": rows.view(T, k).to(torch.int32)}


def _turn(x, cos, sin, rope, rot):
    """x [T, heads, D] rotated by cos, sin [T, rot / 2]."""
    if not rot:
        return x
    cos, sin = cos[:, None], sin[:, None]
    if rope == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _norm(x, weight, eps):
    return x if weight is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def _plain_append(s):
    """Queries in 32 bits, but for the angles; keys in 64, rounded to 32: their codes are asked next to borders."""
    live = s["positions"] >= 0
    rot, cos, sin = 0, None, None
    if s["inv_freq"] is not None:
        rot = 2 * s["inv_freq"].numel()
        angle = s["positions"].double()[:, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle), torch.sin(angle)
    low = (None, None) if cos is None else (cos.float(), sin.float())
    q = _turn(_norm(s["q"].float(), s["q_weight"], s["eps"]), *low, s["rope"], rot).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
    k = _turn(_norm(s["k"].double(), None if s["k_weight"] is None else s["k_weight"].double(), s["eps"]), cos, sin, s["rope"], rot)
    heads, D = s["k"].shape[1:]
    has = live.nonzero().squeeze(1)
    _plain_write(k.float()[has], s["v"][has], s["slots"][has], s["cache"], s["page"])
    k, v = _plain_read(s["cache"], s["slots"][has], heads, D, s["page"])
    s["k_out"][has], s["v_out"][has] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


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


def _blocks(cache, heads, D, page):
    """Views of the four regions of every (page, head) block of a cache."""
    n, m = page // 16, D // 32
    blk = cache.view(-1, heads, page * D * 17 // 16)
    a, b, c = page * D // 2, page * D, page * D + page * m
    return (blk[..., :a].unflatten(-1, (n, m, 16, 16)), blk[..., a:b].unflatten(-1, (n, 4, 16, m, 4)),
            blk[..., b:c].unflatten(-1, (n, m, 16)), blk[..., c:].unflatten(-1, (n, 16, m)))


def _plain_write(k, v, slots, cache, page):
    heads, D = k.shape[1:]
    kc, vc, ks, vs = _blocks(cache, heads, D, page)
    p, t = slots // page, slots % page
    n, r = t // 16, t % 16
    c, s = _quantize(k)
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


def _plain_verify(s):
    """Sums in 64 bits: where a running sum passes a number is asked next to borders."""
    P, Q, tokens, cu = s["target"], s["draft"], s["tokens"], s["cu_q"].long()
    T, V = P.shape
    B = cu.numel() - 1
    n = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=P.device)
    rows = (cu[:-1, None] + i).clamp_max(T - 1)                       # [B, max_q]
    x = tokens.long()[(rows + 1).clamp_max(T - 1)]                    # the draft that each row judges
    p = P[rows, x].double()
    q = torch.ones_like(p) if Q is None else Q[rows, x].double()
    good = (s["accept"][rows].double() * q < p) & (i < n[:, None] - 1)
    acc = torch.cumprod(good.long(), 1).sum(1)
    row = (cu[:-1] + acc).clamp_max(T - 1)
    w = P[row].double()
    refused = tokens.long()[(row + 1).clamp_max(T - 1)]
    if Q is None:
        rest = w.scatter(1, refused[:, None], 0.0)
    else:
        rest = (w - Q[row].double()).clamp_min(0)
    rest = torch.where(((acc < n - 1) & (rest.sum(1) > 0))[:, None], rest, w)
    total = torch.cumsum(rest, 1)
    pick = (total <= s["sample"].double()[:, None] * total[:, -1:]).sum(1).clamp_max(V - 1)
    t = torch.arange(T, device=P.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp_max(B - 1)
    at = t - cu[b]
    out = torch.where(at < acc[b], tokens.long()[(t + 1).clamp_max(T - 1)], torch.where(at == acc[b], pick[b], -1))
    out = torch.where(t < cu[-1], out, -1)
    return {"tokens": out.to(torch.int32), "accepted": acc.to(torch.int32), "lens": (s["kv_lens"] - (n - 1 - acc)).to(torch.int32)}


# ------------------------------------------------------------------------------- what a pass needs

def work(case):
    if case["kind"] == "route":
        live = case["T"] - case["padded"]
        return {"bytes": live * case["E"] * (4 if case["fp32"] else 2) + 8 * case["T"] * case["topk"], "flops": 0}
    if case["kind"] == "sort":
        return {"bytes": 12 * case["T"] * case["topk"] + 4 * case["local"] + 4, "flops": 0}
    if case["kind"] == "append":  # rows in, cache and queries out; cache in, rows out
        live, D, H = case["T"] - case["padded"], case["D"], case["Hkv"]
        return {"bytes": live * (4 * H * case["G"] * D + 8 * H * D + 2 * 2 * H * D * 17 // 32 + 20), "flops": 0}
    n = _rows_of(case)
    each = case["V"] * 4 * (2 if case["sampled"] else 1)  # the row that the next token comes from
    return {"bytes": len(n) * (each + 20) + sum(n) * 20, "flops": 0}


# ------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "sort": _exact_sort, "append": _exact_append, "verify": _exact_verify}[case["kind"]](s)


def _exact_route(s):
    """On the host, a choice at a time over all tokens."""
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    p = np.exp(x - np.logaddexp.reduce(x, axis=1, keepdims=True)) if s["score"] == "softmax" else 0.5 + 0.5 * np.tanh(x / 2)
    left = x.copy() if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    G, all_rows = s["groups"], np.arange(T)
    if G > 1:
        by = left if s["bias"] is not None or s["group_top"] == 1 else p
        v = np.partition(by.reshape(T, G, -1), E // G - s["group_top"], axis=2)[..., E // G - s["group_top"]:].sum(2)
        for g in range(G):  # a group stays if fewer than topk_groups stand before it
            before = (v > v[:, g:g + 1]).sum(1) + (v[:, :g] == v[:, g:g + 1]).sum(1)
            left[before >= s["topk_groups"], g * (E // G):(g + 1) * (E // G)] = -np.inf
    ids = np.empty((T, s["topk"]), dtype=np.int64)
    for j in range(s["topk"]):
        ids[:, j] = left.argmax(1)  # the first of equals
        left[all_rows, ids[:, j]] = -np.inf
    w = np.take_along_axis(p, ids, 1)
    w = s["scale"] * (w / w.sum(1, keepdims=True) if s["renormalize"] else w)
    if s["num_rows"] is not None:
        ids[int(s["num_rows"]):], w[int(s["num_rows"]):] = -1, 0
    return {"ids": torch.from_numpy(ids.astype(np.int32)), "weights": torch.from_numpy(w)}


def _exact_sort(s):
    """Expert by expert on the host."""
    ids = s["ids"].cpu().numpy()
    T, k = ids.shape
    if T * k * s["E"] > 1 << 27:
        return None
    flat = ids.reshape(-1) - s["first"]
    lists = [np.flatnonzero(flat == e) for e in range(s["E"])]
    order = np.concatenate(lists)
    row_token, rows = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
    row_token[:order.size] = order // k
    rows[order] = np.arange(order.size)
    offsets = np.cumsum([0] + [x.size for x in lists]).astype(np.int32)
    return {"offsets": torch.from_numpy(offsets), "row_token": torch.from_numpy(row_token), "token_rows": torch.from_numpy(rows.reshape(T, k))}


def _exact_append(s):
    live = s["positions"] >= 0
    out = {}
    for name, x, w in (("q", s["q"], s["q_weight"]), ("k", s["k"], s["k_weight"])):
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for t in range(0, x.shape[0], 2048):
            at = slice(t, t + 2048)
            z = x[at].double()
            if w is not None:
                z = z * torch.rsqrt(z.square().sum(-1, keepdim=True) / z.shape[-1] + s["eps"]) * w.double()
            if s["inv_freq"] is not None:  # as products of complex numbers
                m = s["inv_freq"].numel()
                turn = torch.outer(s["positions"][at].double(), s["inv_freq"].double())
                turn = torch.complex(torch.cos(turn), torch.sin(turn))[:, None]
                if s["rope"] == "halves":
                    c = torch.complex(z[..., :m], z[..., m:2 * m]) * turn
                    z = torch.cat([c.real, c.imag, z[..., 2 * m:]], -1)
                else:
                    c = torch.view_as_complex(z[..., :2 * m].unflatten(-1, (m, 2)).contiguous()) * turn
                    z = torch.cat([torch.view_as_real(c).flatten(-2), z[..., 2 * m:]], -1)
            y[at] = z if name == "q" else _exact_mx(z)
        out[name] = y
    out["v"] = _exact_mx(s["v"].double())
    return {name: y * live[:, None, None] for name, y in out.items()}


def _exact_mx(x):
    """The nearest E2M1 value, ties to the even code, at the block's power of two; in 64 bits."""
    x = x.unflatten(-1, (-1, 32))
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


def _exact_verify(s):
    """Request by request on the host."""
    cu, kv = s["cu_q"].tolist(), s["kv_lens"].tolist()
    tokens, accept, sample = s["tokens"].tolist(), s["accept"].tolist(), s["sample"].tolist()
    out, accepted, lens = [-1] * len(tokens), [], []
    for b in range(len(kv)):
        t, last = cu[b], cu[b + 1] - 1
        while t < last:
            x = tokens[t + 1]
            if not accept[t] * (1.0 if s["draft"] is None else float(s["draft"][t, x])) < float(s["target"][t, x]):
                break
            out[t] = x
            t += 1
        p = s["target"][t].double().cpu().numpy()
        w = p.copy()
        if t < last:
            if s["draft"] is None:
                w[tokens[t + 1]] = 0
            else:
                w = np.maximum(p - s["draft"][t].double().cpu().numpy(), 0)
            if not w.sum() > 0:
                w = p
        total = np.cumsum(w)
        out[t] = min(int(np.searchsorted(total, sample[b] * total[-1], side="right")), w.size - 1)
        accepted.append(t - cu[b])
        lens.append(kv[b] - (last - t))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"tokens": i32(out), "accepted": i32(accepted), "lens": i32(lens)}
