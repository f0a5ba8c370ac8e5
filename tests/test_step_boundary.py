"""Routing, its tables, the cache's append and the verification of drafts on the host: argument errors
before any HIP call, workspace sizes, and the binding's checks of tensors' metadata. None of these runs
anything on a GPU."""
import os

import pytest

import mxfp4_quantized_gemm_inline_amd as mx

pytestmark = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmxgemm.so not built")

A, B, C, D_, E_, F, G, H = (0x10000 * i for i in range(1, 9))  # fake, aligned addresses
INF, NAN = float("inf"), float("nan")


def _call(name, base, status, **changes):
    args = dict(base)
    args.update(changes)
    assert getattr(mx.lib(), name)(*args.values()) == status, changes


def test_route_argument_errors():
    base = dict(logits=A, stride=64, type=0, bias=B, T=4, E=64, topk=8, score=0, groups=8, keep=4, top=2, renorm=1, scale=1.0, rows=C,
                ids=D_, weights=E_, stream=None)
    for k, v in (("stride", -1), ("stride", 1 << 32), ("type", 2), ("type", -1), ("T", -1), ("T", (1 << 27) + 1), ("E", 0), ("E", -8),
                 ("E", 1025), ("E", 60), ("topk", 0), ("topk", -3), ("topk", 33), ("topk", 65), ("score", 2), ("groups", 0), ("groups", 65), ("groups", 7),
                 ("keep", 0), ("keep", 9), ("top", 0), ("top", 3), ("renorm", 2), ("scale", INF), ("scale", NAN)):
        _call("mx_moe_route", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("logits", "ids", "weights"):
        _call("mx_moe_route", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("bias", "rows", "ids", "weights"):
        _call("mx_moe_route", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_moe_route", base, mx.MX_ERR_ALIGN, logits=0x10001)
    _call("mx_moe_route", base, mx.MX_ERR_ALIGN, logits=0x10002, type=1)
    _call("mx_moe_route", base, mx.MX_OK, T=0, logits=None, ids=None, weights=None)
    _call("mx_moe_route", base, mx.MX_ERR_SHAPE, T=0, topk=0)


def test_sort_argument_errors():
    base = dict(ids=A, T=4, topk=8, first=0, E=64, offsets=B, token=C, rows=D_, ws=None, ws_bytes=0, stream=None)
    for k, v in (("T", -1), ("T", (1 << 25) + 1), ("T", 1 << 62), ("topk", 0), ("topk", 1025), ("first", -1), ("first", 1 << 30), ("E", 0), ("E", 1025)):
        _call("mx_moe_sort", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("ids", "offsets", "token", "rows"):
        _call("mx_moe_sort", base, mx.MX_ERR_NULL, **{k: None})
        _call("mx_moe_sort", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_moe_sort", base, mx.MX_ERR_NULL, T=0, offsets=None)
    _call("mx_moe_sort", base, mx.MX_ERR_ALIGN, ws=0x10008)
    size = mx.mx_moe_sort_workspace_bytes
    assert size(0, 8, 64) == 0 and size(4, 8, 64) == 0 and size(-1, 8, 64) == 0 and size(4, 0, 64) == 0
    big = size(1 << 25, 8, 1024)
    assert 0 < big <= 1025 * 1024 * 4
    _call("mx_moe_sort", base, mx.MX_ERR_WORKSPACE, T=1 << 25, E=1024)
    _call("mx_moe_sort", base, mx.MX_ERR_WORKSPACE, T=1 << 25, E=1024, ws=A, ws_bytes=big - 1)


def test_append_argument_errors():
    base = dict(q=A, qs=1024, k=B, ks=256, v=C, vs=256, pos=D_, slots=E_, T=4, Hq=8, H=2, D=128, cache=F, pages=3, page=16, qw=G, kw=G,
                eps=1e-6, freq=H, rot=128, rope=0, scale=1.0, out=0x90000, os=1024, stream=None)
    for k, v in (("qs", 1020), ("qs", -8), ("qs", 1 << 32), ("ks", 12), ("vs", -8), ("os", 1016), ("os", 1028), ("T", -1), ("T", (1 << 30) + 1), ("Hq", -1),
                 ("Hq", 1025), ("H", -1), ("H", 1025), ("D", 96), ("D", 0), ("pages", 0), ("page", 20), ("rot", -16), ("rot", 8),
                 ("rot", 144), ("rope", 2), ("eps", -1.0), ("eps", INF), ("eps", NAN), ("scale", INF), ("scale", NAN)):
        _call("mx_kv_append", base, mx.MX_ERR_SHAPE, **{k: v})
    _call("mx_kv_append", base, mx.MX_ERR_SHAPE, Hq=0, H=0, pages=0)
    _call("mx_kv_append", base, mx.MX_ERR_SHAPE, H=0)                       # pages without heads
    _call("mx_kv_append", base, mx.MX_ERR_SHAPE, out=A, os=2048)            # in place with another stride
    for k in ("q", "k", "v", "pos", "slots", "cache", "freq", "out"):
        _call("mx_kv_append", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("q", "k", "v", "cache", "out"):
        _call("mx_kv_append", base, mx.MX_ERR_ALIGN, **{k: 0x10008})
    for k in ("pos", "qw", "kw", "freq"):
        _call("mx_kv_append", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_kv_append", base, mx.MX_ERR_ALIGN, slots=0x10004)
    _call("mx_kv_append", base, mx.MX_OK, T=0, q=None)
    # what is not used is not asked for
    _call("mx_kv_append", base, mx.MX_ERR_NULL, Hq=0, q=None, out=None, qs=3, os=3, pos=None)
    _call("mx_kv_append", base, mx.MX_ERR_NULL, H=0, pages=0, k=None, v=None, slots=None, cache=None, ks=3, vs=3, pos=None)


def test_verify_argument_errors():
    base = dict(p=A, ps=100, q=B, qs=100, tokens=C, cu=D_, kv=E_, accept=F, sample=G, T=9, B=3, V=100, out=H, acc=0x90000, lens=0xA0000,
                ws=0xB0000, ws_bytes=1 << 20, stream=None)
    for k, v in (("ps", 99), ("ps", -1), ("ps", 1 << 32), ("qs", 99), ("T", -1), ("T", (1 << 30) + 1), ("B", -1), ("B", (1 << 16) - 1), ("V", 0),
                 ("V", (1 << 24) + 1)):
        _call("mx_verify_drafts", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("p", "tokens", "cu", "kv", "accept", "sample", "out", "acc", "lens"):
        _call("mx_verify_drafts", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("p", "q", "tokens", "cu", "kv", "accept", "sample", "out", "acc", "lens"):
        _call("mx_verify_drafts", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_verify_drafts", base, mx.MX_ERR_ALIGN, ws=0x10008)
    need = mx.mx_verify_drafts_workspace_bytes(3, 100)
    assert need > 0 and mx.mx_verify_drafts_workspace_bytes(0, 100) == 0 and mx.mx_verify_drafts_workspace_bytes(3, 0) == 0
    _call("mx_verify_drafts", base, mx.MX_ERR_WORKSPACE, ws=None)
    _call("mx_verify_drafts", base, mx.MX_ERR_WORKSPACE, ws_bytes=need - 1)
    _call("mx_verify_drafts", base, mx.MX_OK, T=0, B=0, p=None, cu=None)


def test_binding_checks_metadata():
    torch = pytest.importorskip("torch")
    bf, f32, i32, i64, u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8
    l = torch.zeros((5, 64), dtype=bf)
    for error, args, kw in (
            (TypeError, (l.half(), 4), {}), (TypeError, (l.tolist(), 4), {}), (ValueError, (l[0], 4), {}), (ValueError, (l.t(), 4), {}),
            (TypeError, (l, 4), dict(bias=l[0])), (ValueError, (l, 4), dict(bias=torch.zeros(63))),
            (TypeError, (l, 4), dict(num_rows=torch.zeros(1))), (ValueError, (l, 4), dict(ids=torch.zeros((5, 3), dtype=i32))),
            (TypeError, (l, 4), dict(ids=torch.zeros((5, 4), dtype=i64))), (ValueError, (l, 4), dict(weights=torch.zeros((4, 4)))),
            (ValueError, (l, 4), {})):  # a host tensor
        with pytest.raises(error):
            mx.mx_moe_route(*args, **kw)
    ids = torch.zeros((5, 4), dtype=i32)
    for error, args, kw in (
            (TypeError, (ids.long(), 8), {}), (ValueError, (ids[0], 8), {}), (ValueError, (ids[:, :2], 8), {}),
            (ValueError, (ids, 8), dict(expert_offsets=torch.zeros(8, dtype=i32))), (ValueError, (ids, 8), dict(row_token=torch.zeros(19, dtype=i32))),
            (ValueError, (ids, 8), dict(token_rows=torch.zeros((4, 5), dtype=i32))), (ValueError, (ids, 8), {}), (ValueError, (ids, 0), {})):
        with pytest.raises(error):
            mx.mx_moe_sort(*args, **kw)
    q, k = torch.zeros((5, 4, 64), dtype=bf), torch.zeros((5, 2, 64), dtype=bf)
    pos, slots, w = torch.zeros(5, dtype=i32), torch.zeros(5, dtype=i64), torch.ones(64)
    cache = torch.zeros(mx.mx_kv_cache_bytes(2, 16, 2, 64), dtype=u8)
    good = dict(q_bf16=q, k_bf16=k, v_bf16=k, positions=pos, slots=slots, cache=cache, page_size=16)
    for error, kw in (
            (TypeError, dict(q_bf16=q.float())), (TypeError, dict(v_bf16=None)), (ValueError, dict(v_bf16=k[:4])), (ValueError, dict(k_bf16=k[:4])),
            (ValueError, dict(k_bf16=None)), (ValueError, dict(q_bf16=None, k_bf16=None)), (ValueError, dict(q_bf16=None, q_out=q)),
            (TypeError, dict(positions=slots)), (ValueError, dict(positions=pos[:4])), (TypeError, dict(slots=pos)), (TypeError, dict(slots=None)),
            (ValueError, dict(slots=slots[:4])), (ValueError, dict(cache=cache[:100])), (TypeError, dict(cache=None)),
            (TypeError, dict(q_weight=w.to(bf))), (ValueError, dict(k_weight=w[:32])), (TypeError, dict(inv_freq=w.double())),
            (ValueError, dict(q_out=q[:, :2])), (TypeError, dict(q_out=q.float())), (mx.MxError, dict(page_size=24)), (ValueError, {})):
        with pytest.raises(error):
            mx.mx_kv_append(**{**good, **kw})
    p, toks, cu, kv, u = torch.zeros((9, 50)), torch.zeros(9, dtype=i32), torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(9)
    good = [p, p, toks, cu, kv, u, u[:3]]
    for error, i, bad in ((TypeError, 0, p.to(bf)), (ValueError, 0, p.t()), (TypeError, 1, p.double()), (ValueError, 1, p[:, :49]), (ValueError, 1, p[:8]),
                          (TypeError, 2, toks.long()), (ValueError, 2, toks[:8]), (ValueError, 3, cu[:3]), (TypeError, 4, kv.float()),
                          (ValueError, 5, u[:8]), (TypeError, 5, u.double()), (ValueError, 6, u[:2]), (ValueError, 6, u[::4])):
        with pytest.raises(error):
            mx.mx_verify_drafts(*good[:i], bad, *good[i + 1:])
    for kw in (dict(out_tokens=toks[:8]), dict(accepted=kv[:2]), dict(new_lens=kv[:2]), {}):
        with pytest.raises(ValueError):
            mx.mx_verify_drafts(*good, **kw)
