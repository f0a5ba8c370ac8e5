"""The key/value cache calls on the host: sizes, argument errors before any HIP call, plans, and
the binding's checks of tensors' metadata. None of these runs anything on a GPU."""
import os

import pytest

import mxfp4_quantized_gemm_inline_amd as mx

pytestmark = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmxgemm.so not built")

A, B, C, D_, E, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000  # fake, aligned addresses


def test_cache_bytes():
    assert mx.mx_kv_cache_bytes(1, 16, 1, 128) == 16 * 128 * 17 // 16
    assert mx.mx_kv_cache_bytes(1000, 64, 8, 64) == 1000 * 64 * 8 * 64 * 17 // 16
    assert mx.mx_kv_cache_bytes((1 << 31) - 1, 1024, 1024, 256) == ((1 << 31) - 1) * 1024 * 1024 * 272
    for bad in ((0, 16, 1, 128), (1 << 31, 16, 1, 128), (1, 8, 1, 128), (1, 24, 1, 128), (1, 2048, 1, 128), (1, 16, 0, 128),
                (1, 16, 1025, 128), (1, 16, 1, 96), (1, 16, 1, 0), (-1, 16, 1, 64)):
        assert mx.mx_kv_cache_bytes(*bad) == 0, bad


def _call(name, base, status, **changes):
    args = dict(base)
    args.update(changes)
    assert getattr(mx.lib(), name)(*args.values()) == status, changes


def test_tables_argument_errors():
    base = dict(old=A, new=B, B=4, page=16, table=C, blocks=8, stack=D_, capacity=10, count=E, count_out=F, rows=8, cu=A,
                slots=B, pos=C, flag=D_, ws=None, ws_bytes=0, stream=None)
    for k, v in (("B", -1), ("B", (1 << 20) + 1), ("page", 15), ("page", 48), ("page", 2048), ("blocks", 0),
                 ("blocks", (1 << 26) + 1), ("capacity", -1), ("capacity", 1 << 31), ("rows", -1), ("rows", (1 << 30) + 1)):
        _call("mx_kv_tables", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("old", "new", "table", "stack", "count", "count_out", "cu", "slots", "pos", "flag"):
        _call("mx_kv_tables", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("old", "new", "table", "stack", "count", "count_out", "cu", "pos", "flag"):
        _call("mx_kv_tables", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_kv_tables", base, mx.MX_ERR_ALIGN, slots=0x10004)
    _call("mx_kv_tables", base, mx.MX_ERR_ALIGN, ws=0x10008)
    assert mx.mx_kv_tables_workspace_bytes(4, 8) == 0
    need = mx.mx_kv_tables_workspace_bytes(5000, 100)
    assert need >= 3 * 4 * 5001
    assert mx.mx_kv_tables_workspace_bytes(4, 1 << 20) > 0 and mx.mx_kv_tables_workspace_bytes(-1, 8) == 0
    _call("mx_kv_tables", base, mx.MX_ERR_WORKSPACE, B=5000)
    _call("mx_kv_tables", base, mx.MX_ERR_WORKSPACE, B=5000, ws=A, ws_bytes=need - 1)


def test_write_and_read_argument_errors():
    base = dict(k=A, ks=256, v=B, vs=256, slots=C, T=4, cache=D_, pages=3, page=16, heads=2, D=128, stream=None)
    for k, v in (("ks", 12), ("vs", -8), ("T", -1), ("T", (1 << 30) + 1), ("pages", 0), ("page", 20), ("heads", 0),
                 ("D", 32), ("ks", 1 << 32)):
        _call("mx_kv_write", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("k", "v", "slots", "cache"):
        _call("mx_kv_write", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("k", "v", "cache"):
        _call("mx_kv_write", base, mx.MX_ERR_ALIGN, **{k: 0x10008})
    _call("mx_kv_write", base, mx.MX_ERR_ALIGN, slots=0x10004)
    _call("mx_kv_write", base, mx.MX_OK, T=0, k=None)
    base = dict(cache=A, pages=3, page=16, heads=2, D=128, slots=B, T=4, k=C, v=D_, stream=None)
    for k, v in (("T", -1), ("pages", 0), ("page", 20), ("heads", 0), ("D", 32)):
        _call("mx_kv_read", base, mx.MX_ERR_SHAPE, **{k: v})
    for k in ("k", "v", "slots", "cache"):
        _call("mx_kv_read", base, mx.MX_ERR_NULL, **{k: None})
        _call("mx_kv_read", base, mx.MX_ERR_ALIGN, **{k: 0x10004})
    _call("mx_kv_read", base, mx.MX_OK, T=0)


def test_attention_argument_errors():
    base = dict(q=A, qs=1024, cache=B, pages=9, page=16, table=C, blocks=4, cu=D_, kv=E, B=2, T=5, Hq=8, H=2, D=128, max_q=3,
                max_kv=60, causal=1, window=0, scale=0.1, out=F, os=1024, ws=None, ws_bytes=0, stream=None)
    for k, v in (("qs", 1020), ("qs", -8), ("os", 1016), ("os", 1028), ("pages", 0), ("page", 17), ("blocks", 0),
                 ("blocks", (1 << 26) + 1), ("B", -1), ("B", (1 << 20) + 1), ("T", -1), ("T", 1 << 30), ("Hq", 9), ("Hq", 0),
                 ("H", 0), ("D", 96), ("max_q", 0), ("max_kv", 0), ("causal", 2), ("window", -1), ("scale", 0.0),
                 ("scale", -1.0), ("scale", float("nan")), ("scale", float("inf"))):
        _call("mx_kv_attention", base, mx.MX_ERR_SHAPE, **{k: v})
    _call("mx_kv_attention", base, mx.MX_ERR_SHAPE, causal=0, window=4)
    for k in ("q", "cache", "table", "cu", "kv", "out"):
        _call("mx_kv_attention", base, mx.MX_ERR_NULL, **{k: None})
    for k in ("q", "cache", "out", "ws"):
        _call("mx_kv_attention", base, mx.MX_ERR_ALIGN, **{k: 0x10008})
    for k in ("table", "cu", "kv"):
        _call("mx_kv_attention", base, mx.MX_ERR_ALIGN, **{k: 0x10002})
    _call("mx_kv_attention", base, mx.MX_OK, T=0, q=None)
    _call("mx_kv_attention", base, mx.MX_OK, B=0, q=None)
    assert mx.mx_kv_attention_plan(2, 0, 8, 2, 128, 1, 64) == "none"
    with pytest.raises(mx.MxError):
        mx.mx_kv_attention_plan(2, 5, 9, 2, 128, 1, 64)
    assert mx.lib().mx_kv_attention_plan(2, 5, 8, 2, 128, 1, 64, 0, 0, None, 0) == mx.MX_ERR_NULL


def test_attention_plan_follows_rows_and_lengths():
    plan, ws = mx.mx_kv_attention_plan, mx.mx_kv_attention_workspace_bytes
    # decoding: equal shares of the tokens, more of them where there are many segments of 64 elements
    assert plan(64, 64, 64, 8, 128, 1, 8192) == "k_kv_attn_few<128, 1, true> workers=512 + k_kv_attn_seams"
    assert plan(512, 512, 64, 8, 128, 1, 20000) == "k_kv_attn_few<128, 1, true> workers=512 + k_kv_attn_seams"
    assert plan(64, 64, 64, 8, 64, 1, 8192) == "k_kv_attn_few<64, 1, true> workers=1024 + k_kv_attn_seams"
    assert plan(8, 8, 64, 8, 64, 1, 8192) == "k_kv_attn_few<64, 1, true> workers=512 + k_kv_attn_seams"
    assert ws(64, 64, 64, 8, 128, 1, 8192) == 512 * (2 * 16 * (128 + 2) * 4 + 16)
    # short segments, also by a window, and very many of them, stay whole
    assert plan(512, 512, 64, 8, 128, 1, 2048) == "k_kv_attn_few<128, 1, false>"
    assert plan(32, 128, 12, 12, 64, 4, 4001, 1024) == "k_kv_attn_few<64, 1, false>"
    assert plan(256, 256, 64, 8, 128, 1, 700) == "k_kv_attn_few<128, 1, false>"
    assert ws(256, 256, 64, 8, 128, 1, 700) == 0
    # tiles of up to 32 rows, 16 at D = 256
    assert plan(4, 16, 32, 4, 128, 4, 100).startswith("k_kv_attn_few<128, 2, false>")
    assert plan(4, 16, 32, 4, 256, 4, 100) == "k_kv_attn_few<256, 1, false>"
    # more rows: by the longest request's and the average
    assert plan(64, 512, 32, 4, 128, 8, 100) == "k_kv_attn_few<128, 2, false>"
    assert plan(64, 1024, 32, 4, 128, 16, 100) == "k_kv_attn_many<128> C=128 S=1"
    assert plan(64, 500, 32, 4, 128, 17, 100) == "k_kv_attn_few<128, 1, false> + k_kv_attn_many<128> C=128 S=1"
    assert plan(64, 500, 80, 4, 256, 17, 100) == "k_kv_attn_many<256> C=128 S=1"
    # whole prompts fill the chip; few tiles over a long cache are split
    assert plan(1, 8192, 32, 8, 128, 8192, 8192) == "k_kv_attn_many<128> C=8192 S=1"
    assert plan(1, 512, 32, 8, 128, 512, 16000) == "k_kv_attn_many<128> C=4032 S=4 + k_kv_attn_join"
    assert ws(1, 512, 32, 8, 128, 512, 16000) == 512 * 32 * (4 * 130 + 1) * 4
    # rows of both kinds: each kernel its own; without the workspace neither cuts
    assert plan(20, 1553, 32, 4, 128, 512, 4096) == ("k_kv_attn_few<128, 1, true> workers=512 + k_kv_attn_seams + "
                                                     "k_kv_attn_many<128> C=4096 S=1")
    assert plan(20, 1553, 32, 4, 128, 512, 4096, workspace_bytes=0) == ("k_kv_attn_few<128, 1, false> + "
                                                                       "k_kv_attn_many<128> C=1073741824 S=1")
    for hint in (1, 10 ** 6, 2 ** 62):
        assert plan(3, 7, 8, 2, 64, hint, hint, 2 ** 62) != ""


def test_binding_checks_metadata():
    torch = pytest.importorskip("torch")
    bf, i32, i64, u8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8
    k = torch.zeros((5, 2, 64), dtype=bf)
    cache = torch.zeros(mx.mx_kv_cache_bytes(2, 16, 2, 64), dtype=u8)
    slots = torch.zeros(5, dtype=i64)
    with pytest.raises(TypeError):
        mx.mx_kv_write(k.float(), k, slots, cache, 16)
    with pytest.raises(TypeError):
        mx.mx_kv_write(k, k, slots.int(), cache, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_write(k, k[:4], slots, cache, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_write(k, k, slots[:4], cache, 16)
    with pytest.raises(ValueError):       # heads are not dense
        mx.mx_kv_write(k.transpose(1, 2).contiguous().transpose(1, 2), k, slots, cache, 16)
    with pytest.raises(ValueError):       # less than one page
        mx.mx_kv_write(k, k, slots, cache[:100], 16)
    with pytest.raises(mx.MxError):
        mx.mx_kv_write(k, k, slots, cache, 24)
    with pytest.raises(ValueError):       # host tensors
        mx.mx_kv_write(k, k, slots, cache, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_read(cache, slots, 2, 64, 16, k_out=torch.zeros((4, 2, 64), dtype=bf))
    table, lens = torch.zeros((3, 4), dtype=i32), torch.zeros(3, dtype=i32)
    stack, one = torch.zeros(6, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError):
        mx.mx_kv_tables(lens[:2], lens, table, stack, one, 16, 8)
    with pytest.raises(TypeError):
        mx.mx_kv_tables(lens, lens.long(), table, stack, one, 16, 8)
    with pytest.raises(ValueError):
        mx.mx_kv_tables(lens, lens, table, stack, one, 16, 8, slots=torch.zeros(7, dtype=i64))
    with pytest.raises(ValueError):
        mx.mx_kv_tables(lens, lens, table, stack, one, 16, 8)
    q, cu = torch.zeros((5, 4, 64), dtype=bf), torch.zeros(4, dtype=i32)
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, table, cu[:3], lens, 2, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, table, cu, lens[:2], 2, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, table, cu, lens, 2, 16, out=torch.zeros((5, 4, 32), dtype=bf))
    with pytest.raises(TypeError):
        mx.mx_kv_attention(q.half(), cache, table, cu, lens, 2, 16)
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, table, cu, lens, 2, 16, workspace=False)
