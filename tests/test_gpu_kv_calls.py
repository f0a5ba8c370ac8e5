"""Calls of the key/value cache as programs make them: on a stream of their own, with workspaces of any
size, with as many heads as the calls take."""
import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_kv import Case, _close, dev
from test_gpu_kv_masks import plan_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T_extra", [(5, 3), (1500, 0)])
def test_every_call_on_another_stream(B, T_extra):
    """Tables, write, read and attention one after the other on a side stream, each allocating its own
    outputs and workspace there, three times over; the current stream stays busy with allocations."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    H, G, D, page, width = 1, 2, 64, 16, 3
    rng = np.random.default_rng(B)
    side = torch.cuda.Stream()
    for again in range(3):
        new = rng.integers(0, width * page + 1, B).astype(np.int32)
        new[0] = width * page
        old = np.zeros(B, np.int32)
        rows, pages = int(new.sum()) + T_extra, int((-(-new // page)).sum())
        table, stack = np.full((B, width), -1, np.int32), rng.permutation(pages).astype(np.int32)
        want = KV.tables(old, new, table, stack, pages, page, rows)
        k, v, q = (W.normal_bf16((rows, n, D), seed=again + 10 * n) for n in (H, H + 1, H * G))
        v = np.ascontiguousarray(v[:, :H])
        args = [dev(x) for x in (old, new, table, stack, np.array([pages], np.int32))]
        kd, vd, qd = dev_bf16(k), dev_bf16(v), dev_bf16(q)
        cache = torch.full((pages, H, KV.block_bytes(page, D)), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        cu, slots, pos, after, status = mx.mx_kv_tables(*args, page, rows, stream=side)
        mx.mx_kv_write(kd, vd, slots, cache, page, stream=side)
        kr, vr = mx.mx_kv_read(cache, slots, H, D, page, stream=side)
        out = mx.mx_kv_attention(qd, cache, args[2], cu, args[1], H, page, max_q=width * page, max_kv=width * page, stream=side)
        for _ in range(8):
            torch.full((1 << 20,), 3, dtype=torch.int32, device="cuda")  # must not take the calls' memory
        side.synchronize()
        for got, w in zip((cu, slots, pos), want):
            assert np.array_equal(got.cpu().numpy(), w)
        assert int(status[0]) == 0 and int(after[0]) == want[3] == 0
        n = int(want[0][-1])
        host = np.full(tuple(cache.shape), 255, np.uint8)
        KV.write(host, k, v, want[1], page)
        assert np.array_equal(cache.cpu().numpy(), host)
        wk, wv = KV.read(host, want[1][:n], page, D)
        assert np.array_equal(O.bf16_to_f64(host_bits(kr))[:n], wk) and np.array_equal(O.bf16_to_f64(host_bits(vr))[:n], wv)
        some = [0, B // 2, B - 1]                      # the oracle is slow over thousands of requests
        for b in some:
            r0, r1 = int(want[0][b]), int(want[0][b + 1])
            exact, bound = KV.attention(O.bf16_to_f64(q[r0:r1]), host, want[5][b:b + 1], [0, r1 - r0], [int(new[b])], page, True, 0,
                                        D ** -0.5)
            _close(host_bits(out)[r0:r1], exact, bound, f"request {b}")


@pytest.mark.parametrize("D,H,G,q,kv", [(64, 2, 4, [1] * 6, [3000, 900, 1, 0, 2000, 77]), (128, 2, 8, [4, 4, 4], [3000, 90, 1500]),
                                        (256, 1, 2, [1, 1], [2500, 1900]), (64, 1, 1, [150, 2], [3000, 1300]),
                                        (128, 1, 2, [150, 2], [3000, 1300]), (256, 1, 1, [150, 2], [3000, 1300])])
def test_workspaces_of_every_size_and_nothing_past_them(D, H, G, q, kv):
    """All that is asked for, a byte less, what one kernel needs, next to nothing: right, and the bytes
    behind the workspace keep what they held."""
    torch = torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, 32, q, kv, seed=D + H)
    need = mx.mx_kv_attention_workspace_bytes(len(q), c.T, H * G, H, D, max(q), max(kv))
    assert need > 0
    plans = set()
    for nbytes in (need + 512, need, need - 1, need // 2, need // 16, 16, 0):
        home = torch.full((nbytes + 4096,), 171, dtype=torch.uint8, device="cuda")
        plans.add(mx.mx_kv_attention_plan(len(q), c.T, H * G, H, D, max(q), max(kv), workspace_bytes=nbytes))
        c.check(mx, what=f"{nbytes} of {need} bytes", workspace=home[:nbytes])
        assert bool((home[nbytes:] == 171).all()), f"past {nbytes} of {need} bytes"
    assert len(plans) >= 2, plans


@pytest.mark.parametrize("D,H,G,q,kv", [(64, 200, 1, [1, 2], [70, 300]), (64, 1024, 1, [1], [40]), (64, 1, 1024, [1, 2], [70, 33]),
                                        (128, 3, 300, [1], [700]), (256, 48, 1, [1], [1500]), (128, 100, 1, [130], [150])])
def test_as_many_heads_as_a_call_takes(D, H, G, q, kv):
    torch_or_skip()
    mx = lib_or_fail()
    c = Case(D, H, G, 16, q, kv, seed=H + G)
    c.check(mx, what=plan_of(mx, c))
