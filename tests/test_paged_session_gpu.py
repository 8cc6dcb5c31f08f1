"""What a PagedSession keeps and lets go: workspaces, page pools, and the
buffers that captured calls hold."""
import gc
import weakref

import numpy as np
import pytest
import torch

import paged_ref as P
import test_paged_gpu as T
from adaptive_head_kv_gb300 import fastgen as fg
from adaptive_head_kv_gb300.session import PagedSession, make_params

pytestmark = pytest.mark.gpu

B, L, H, N, D = 2, 2, 4, 200, 64
G = B * L * H


def session(max_new=600, **kw):
    p = make_params(B, L, H, N, D, "bf16", 0.9, 0.3, 0.3)
    return PagedSession(p, T.SPECIAL, T.PUNCT, max_new, rope=fg.Rope(T.table(D)[1]), **kw)


def prompt(seed):
    g = T.gen(seed)
    return [T.dev(torch.randn(G, N, D, generator=g).to(torch.bfloat16)) for _ in range(3)] + [
        T.dev(torch.randint(100, 300, (B, N), generator=g, dtype=torch.int32))]


def turn(seed, m):
    g = T.gen(seed)
    return [T.dev(torch.randn(G, m, D, generator=g).to(torch.bfloat16)) for _ in range(2)] + [
        T.dev(torch.randint(100, 300, (B, m), generator=g, dtype=torch.int32))]


def dev_pos(t):
    return T.dev([t] * B, torch.int32)


def same_caches(a, b):
    assert torch.equal(a.cache.rows, b.cache.rows)
    x, y = P.GpuPages(a.cache), P.GpuPages(b.cache)
    for c in range(G):
        for ring, count in ((False, int(x.rows[c])), (True, int(x.caches[c][1]))):
            if count:
                u, v = x.segment(c, ring, count), y.segment(c, ring, count)
                for key in u:
                    assert np.array_equal(u[key], v[key], equal_nan=True), (c, ring, key)


def test_outgrown_workspaces_go_unless_a_captured_call_holds_them():
    s = session()
    s.prefill_with_policy(*prompt(1), torch.full((G,), 4, dtype=torch.int8))
    at, dead = N, []
    for m in (2, 30, 100):  # each needs a larger workspace
        s.append(*turn(m, m), at)
        at += m
        dead.append(weakref.ref(s.aws))
        old = s.dws
        s.reschedule()
        if s.dws is not old:
            dead.append(weakref.ref(old))
    del old
    gc.collect()
    assert [w() is None for w in dead[:2]] == [True, True]
    assert sum(w() is not None for w in dead) <= 2  # the two of now
    pos, x = T.dev([at] * B, torch.int32), turn(9, 100)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.append(*x, pos)
    held = weakref.ref(s.aws)
    s.append(*turn(3, 260), dev_pos(-1))
    gc.collect()
    assert held() is not None and held() is not s.aws
    graph.replay()
    torch.cuda.synchronize()
    other = session()
    other.prefill_with_policy(*prompt(1), torch.full((G,), 4, dtype=torch.int8))
    at = N
    for m in (2, 30, 100):
        other.append(*turn(m, m), at)
        at += m
    other.append(*x, at)
    same_caches(s, other)
    assert int(s.dev_err) == 0


@pytest.mark.parametrize("own_stream", [False, True])
def test_calls_captured_on_a_pool_that_was_replaced_do_nothing_and_say_so(own_stream):
    """A second prompt wants more pages.  Replays of append and decode captured before touch neither
    the memory that the old pool had nor the new cache, and the error word says so; the session's
    own calls go on."""
    stream = torch.cuda.Stream() if own_stream else None
    few, full = torch.zeros(G, dtype=torch.int8), torch.full((G,), 4, dtype=torch.int8)
    s, fresh = session(100, stream=stream), session(100, stream=stream)
    torch.cuda.synchronize()
    s.prefill_with_policy(*prompt(1), few)
    torch.cuda.synchronize()
    short, long_, pos = turn(2, 4), turn(3, 20), dev_pos(N)
    q = T.dev(torch.randn(G, D, generator=T.gen(5)).to(torch.bfloat16))
    one = [x[:, 0].contiguous() for x in turn(4, 1)]
    s.append(*long_, dev_pos(-1))  # sizes the workspace
    out = torch.full((G, D), 3.5, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: s.append(*short, pos), lambda: s.append(*long_, pos),
                 lambda: s.decode(q, *one, pos, out=out)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            call()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert int(s.dev_err) == 0
    pool, before = s.cache.c.n_pages, s.cache
    freed = [s.cache.k_pages.data_ptr(), s.cache.v_pages.data_ptr()]
    for x in (s, fresh):
        x.prefill_with_policy(*prompt(6), full)
        torch.cuda.synchronize()
    assert s.cache.c.n_pages > pool and s.cache is not before
    assert before.k_pages is None and s.cache.k_pages.data_ptr() not in freed
    torch.cuda.synchronize()
    other = [torch.full((pool * 64 * D,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for g in graphs:
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert fg.fastgen_read_error(s.dev_err) == fg.FG_EINVAL
            s.dev_err.zero_()
    assert all(bool((x == 0xA5).all()) for x in other) and bool((out == 3.5).all())
    same_caches(s, fresh)
    outs = []
    for x in (s, fresh):
        x.append(*short, N)
        torch.cuda.synchronize()
        outs.append(x.decode(q, *one, dev_pos(N + 4)).clone())
        torch.cuda.synchronize()
    assert torch.equal(*outs) and int(s.dev_err) == 0
    same_caches(s, fresh)


def test_a_larger_pool_without_captured_calls_replaces_the_old_one():
    s = session(100)
    s.prefill_with_policy(*prompt(1), torch.zeros(G, dtype=torch.int8))
    old, cache = weakref.ref(s.cache.k_pages), s.cache
    s.prefill_with_policy(*prompt(6), torch.full((G,), 4, dtype=torch.int8))
    gc.collect()
    assert old() is None and s.cache is cache


@pytest.mark.parametrize("host", [False, True])
def test_rotation_of_the_callers_tensors(host):
    """in_place: the same caches without a second pair of queries and keys."""
    pol = torch.arange(G, dtype=torch.int8) % 5
    a, b = session(), session(in_place=True)
    kept = [x.clone() for x in prompt(1)]
    for s in (a, b):
        x = [y.clone() for y in kept]
        if host:
            h = [y.cpu().pin_memory() for y in kept]
            s.prefill_host(*h, *x)
        else:
            s.prefill_with_policy(*x, pol)
        torch.cuda.synchronize()
        same = [torch.equal(u, v) for u, v in zip(x, kept)]
        assert same == [s is a, s is a, True, True]
        if s is b:
            assert b._rotated is None
            assert torch.equal(x[0], a._rotated[0]) and torch.equal(x[1], a._rotated[1])
    assert torch.equal(a.policy, b.policy)
    same_caches(a, b)


@pytest.mark.parametrize("which", ["default", "side"])
def test_streams_given_as_addresses(which):
    """A session on a raw stream address: buffers that grow, captured calls, int positions."""
    side = torch.cuda.Stream()
    address = 0 if which == "default" else side.cuda_stream
    pol = torch.full((G,), 4, dtype=torch.int8)
    a, b = session(), session(stream=address)
    outs = []
    q = T.dev(torch.randn(G, D, generator=T.gen(5)).to(torch.bfloat16))
    one = [x[:, 0].contiguous() for x in turn(4, 1)]
    for s in (a, b):
        torch.cuda.synchronize()
        s.prefill_with_policy(*prompt(1), pol)
        at = N
        for m in (2, 30, 100):
            torch.cuda.synchronize()
            s.append(*turn(m, m), at)
            at += m
        s.reschedule()
        torch.cuda.synchronize()
        outs.append(s.decode(q, *one, at).clone())
        torch.cuda.synchronize()
        outs[-1] = s.out.clone()
    assert torch.equal(*outs) and int(b.dev_err) == 0
    same_caches(a, b)
    if which == "side":
        pos = dev_pos(at + 1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.decode(q, *one, pos)
        assert any(x is b.dws for x in b._held)
        graph.replay()
        torch.cuda.synchronize()
        a.decode(q, *one, pos)
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out)
        same_caches(a, b)
