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
