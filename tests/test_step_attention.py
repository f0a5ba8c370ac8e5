"""Append's queries and the attention over the cache it fills, in the steps of tests/test_gpu_step.py's Loop:
the bf16 queries are held to their own bound, the attention to that of those very queries. The CPU
test shows that these bounds tell right queries from wrong ones: not normed, normed without their weight,
rotated by a position that is off by one."""
from types import SimpleNamespace

import numpy as np
import pytest

import workloads as W
from oracle import mx_kv_oracle as KV
from oracle import mx_oracle as O
from oracle import mx_step_oracle as S

from gpu_util import dev_bf16, host_bits, lib_or_fail, torch_or_skip
from test_gpu_step import Loop, dev

STEPS, EPS = 6, 1e-6


def _host_steps(L, stack, freq, qw, kw):
    """The loop's steps by the oracles: what stands in the tables and the cache at each attention."""
    page, H = L.page, L.H
    Hq = H * L.G
    table, count = np.full((L.B, L.width), -1, np.int32), L.pages
    cache, lens = np.full((L.pages, H, KV.block_bytes(page, L.D)), 255, np.uint8), np.zeros(L.B, np.int32)
    for step in range(STEPS):
        qkv, p, q, tokens, accept, sample = Loop.inputs(L, step)
        new = lens + L.n
        cu, slots, pos, count, st, table, stack = KV.tables(lens, new, table, stack, count, page, L.T)
        assert st == 0
        S.append(cache, O.bf16_to_f64(qkv[:, Hq:Hq + H]), qkv[:, Hq + H:], pos, slots, page, kw, EPS, freq, False)
        yield SimpleNamespace(qkv=qkv, rest=(p, q, tokens, accept, sample), q=O.bf16_to_f64(qkv[:, :Hq]), pos=pos, cu=cu, new=new, table=table,
                              cache=cache, live=int(cu[-1]))
        lens = S.verify(p, q, tokens, cu, new, accept, sample)[2]
        _, _, _, count, st, table, stack = KV.tables(new, lens, table, stack, count, page, 0)
        assert st == 0


def _queries_off(bits, x, qw, freq):
    """Which elements of the queries (bf16 bits) are past their bound."""
    y, size = S.norm_rotate(x.q, x.pos, qw, EPS, freq, False)
    return (np.abs(O.bf16_to_f64(bits) - y) > S.query_bound(y, size))[:x.live]


def _attention_of(bits, x, L):
    """(exact, bound) of the attention of the queries with these bf16 bits."""
    return KV.attention(O.bf16_to_f64(bits)[:x.live], x.cache, x.table, x.cu, x.new, L.page, True, 0, L.D ** -0.5)


def _to_bf16(y):
    return W.f32_to_bf16_bits(y.astype(np.float32))


def test_the_bounds_tell_wrong_queries():
    B, drafts, H, G, D, page, width = 5, 3, 2, 4, 64, 16, 6
    L = SimpleNamespace(B=B, n=drafts + 1, H=H, G=G, D=D, page=page, V=300, width=width, T=B * (drafts + 1) + 2, pages=B * width)
    rng = np.random.default_rng(0)
    stack = rng.permutation(L.pages).astype(np.int32)
    freq = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    qw, kw = ((1 + 0.2 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
    ones = np.ones(D, np.float32)
    for x in _host_steps(L, stack, freq, qw, kw):
        made = {"right": S.norm_rotate(x.q, x.pos, qw, EPS, freq, False)[0], "no norm": S.norm_rotate(x.q, x.pos, None, EPS, freq, False)[0],
                "no weight": S.norm_rotate(x.q, x.pos, ones, EPS, freq, False)[0],
                "one position on": S.norm_rotate(x.q, x.pos + 1, qw, EPS, freq, False)[0], "zero": 0 * x.q}
        bits = {name: _to_bf16(y) for name, y in made.items()}
        exact, bound = _attention_of(bits["right"], x, L)
        assert not _queries_off(bits["right"], x, qw, freq).any()
        for name in list(made)[1:]:
            assert _queries_off(bits[name], x, qw, freq).mean() > 0.5, name
            # and an attention that took such queries is seen at once
            wrong, _ = _attention_of(bits[name], x, L)
            assert (np.abs(wrong - exact) > bound).any(), name


@pytest.mark.gpu
def test_queries_and_attention_of_steps_with_drafts():
    torch_or_skip()
    mx = lib_or_fail()

    class Recording:
        def __getattr__(self, name):
            return getattr(mx, name)

        def mx_kv_append(self, *args, **kw):
            self.queries = mx.mx_kv_append(*args, **kw)
            return self.queries

    calls = Recording()
    L = Loop(calls)
    freq, qw, kw = (t.cpu().numpy() for t in (L.freq, L.qw, L.kw))
    for step, x in enumerate(_host_steps(L, L.stack.cpu().numpy(), freq, qw, kw)):
        o = L.step(dev_bf16(x.qkv), *(dev(t) for t in x.rest))[0]
        assert np.array_equal(L.cache.cpu().numpy(), x.cache), step
        bits = host_bits(calls.queries)
        bits[x.live:] = 0  # rows of padding are not written
        assert not _queries_off(bits, x, qw, freq).any(), step
        exact, bound = _attention_of(bits, x, L)
        err = np.abs(O.bf16_to_f64(host_bits(o)[:x.live]) - exact)
        assert np.all(err <= bound), (step, float((err - bound).max()))
