"""Calls of the key/value cache that the library refuses on the host, and what its host functions
answer for unusual arguments. None of these runs anything on a GPU."""
import os

import pytest

import mxfp4_quantized_gemm_inline_amd as mx

pytestmark = pytest.mark.skipif(not os.path.exists(mx.LIB_PATH), reason="libmxgemm.so not built")


def attention_status(**changes):
    args = dict(q=0x10000, qs=1024, cache=0x20000, pages=9, page=16, table=0x30000, blocks=4, cu=0x40000, kv=0x50000, B=2, T=5,
                Hq=8, H=2, D=128, max_q=3, max_kv=60, causal=1, window=0, scale=0.1, out=0x60000, os=1024, ws=None, ws_bytes=0,
                stream=None)
    args.update(changes)
    return mx.lib().mx_kv_attention(*args.values())


def test_attention_scale_ends():
    """The kernels multiply scores by scale * log2 e, which has to be finite in FP32. T == 0 shows that
    a scale inside the range passes the check without a launch."""
    for scale in (2.0 ** -149, 2.0 ** -126, 1.0, 2.0 ** 127):
        assert attention_status(scale=scale, T=0) == mx.MX_OK, scale
    for scale in (2.0 ** 127 * (1 + 2.0 ** -23), 2.5e38, 3.4e38, float("inf"), float("nan"), 0.0, -0.5):
        assert attention_status(scale=scale, T=0) == mx.MX_ERR_SHAPE, scale


def test_workspace_sizes_follow_their_arguments_values():
    """Whole numbers in any type that int() takes, also one whose value changes between two calls."""
    torch = pytest.importorskip("torch")
    n = torch.tensor(5000)
    assert mx.mx_kv_tables_workspace_bytes(n, 100) == mx.mx_kv_tables_workspace_bytes(5000, 100) > 0
    n.fill_(4)
    assert mx.mx_kv_tables_workspace_bytes(n, 100) == 0
    n.fill_(8192)
    long = mx.mx_kv_attention_workspace_bytes(64, 64, 64, 8, 128, 1, n)
    assert long == mx.mx_kv_attention_workspace_bytes(64, 64, 64, 8, 128, 1, 8192) > 0
    n.fill_(100)
    assert mx.mx_kv_attention_workspace_bytes(64, 64, 64, 8, 128, 1, n) == 0


def test_a_workspace_that_is_no_tensor_is_a_type_error():
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    cache = torch.zeros(mx.mx_kv_cache_bytes(2, 16, 2, 64), dtype=torch.uint8)
    table, lens, cu = torch.zeros((3, 4), dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32)
    for bad in (4096, "none", True):
        with pytest.raises(TypeError):
            mx.mx_kv_attention(q, cache, table, cu, lens, 2, 16, workspace=bad)
        with pytest.raises(TypeError):
            mx.mx_kv_tables(lens, lens, table, torch.zeros(6, dtype=i32), torch.zeros(1, dtype=i32), 16, 1 << 20, workspace=bad)
    with pytest.raises(ValueError):
        mx.mx_kv_attention(q, cache, table, cu, lens, 2, 16, workspace=torch.zeros((8, 64))[:, ::2])


def test_attention_plan_without_the_hint_of_rows():
    """max_q defaults to T: right for one request, further launches and workspace for a batch of rows."""
    plan, ws = mx.mx_kv_attention_plan, mx.mx_kv_attention_workspace_bytes
    assert plan(64, 64, 64, 8, 128, 64, 8192) == ("k_kv_attn_few<128, 1, true> workers=512 + k_kv_attn_seams + "
                                                  "k_kv_attn_many<128> C=512 S=16 + k_kv_attn_join")
    assert ws(64, 64, 64, 8, 128, 64, 8192) == ws(64, 64, 64, 8, 128, 1, 8192) + 64 * 64 * (16 * 130 + 1) * 4
    # one request: 8 heads of 2400 rows in tiles of 128 are 150 groups, three times which fit the chip
    assert plan(1, 300, 64, 8, 128, 300, 8192) == "k_kv_attn_many<128> C=2752 S=3 + k_kv_attn_join"
