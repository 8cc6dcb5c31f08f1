"""Descriptors, row counts and pools of paged 8-bit caches that the caller lays
out or changes: what the header says of them holds for every call."""
import pytest
import torch

import paged_ref as P
import test_paged_gpu as T
from adaptive_head_kv_gb300 import fastgen as fg

pytestmark = pytest.mark.gpu


def larger_ring(s, c, w):
    """Cache c's descriptor says w slots, with pages of the pool for all of them."""
    first, spare = int(s.cache.c.table_len) - 4, s.info.max_pages
    s.set_pages(spare + 4)
    s.cache.page_table[first:] = torch.arange(spare, spare + 4, dtype=torch.int32, device="cuda")
    s.cache.caches[c, 1] = w
    s.cache.caches[c, 4] = first
    s.cache.caches[c, 5] = (w + 63) // 64


def flagged(s):
    got = fg.fastgen_read_error(s.err)
    s.err.zero_()
    return got == fg.FG_EINVAL


@pytest.mark.parametrize("r_l", [0.3, 0.0])
@pytest.mark.parametrize("w", [60, 128, -5])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_a_ring_larger_than_the_window_is_flagged_by_every_call(w, r_l, dtype, d):
    """The window is 27 or none.  A descriptor of more slots, with or without more pages: each call
    flags it, reads and writes no row of it, and serves the other caches."""
    def setup():
        s = T.Setup(50, L=1, H=5, n=90, r_l=r_l, dtype=dtype, d=d, max_new=400)
        larger_ring(s, 3, w)
        s.ref[3].w = 0
        return s

    def rest(s):
        gpu = P.GpuPages(s.cache)
        pages = gpu.pages(3, True)[: max(0, -(-w // 64))]
        assert (gpu.pos[pages] == -3).all() and (gpu.codes["k"][pages] == 0.8125).all()
        s.cache.caches[3, 1] = 0  # for the comparison, which reads the descriptor's w
        s.check(empty=False)
        s.cache.caches[3, 1] = w

    s = setup()
    s.compact()
    assert flagged(s)
    rest(s)
    at = 90
    for m in (1, 8, 9, 70):
        ids, k, v = s.tokens(m, m)
        s.append(ids, k, v, [at])
        assert flagged(s), m
        s.ref_append(ids, k, v, [at])
        rest(s)
        at += m
    for again in (False, True):
        if again:
            s.cache.schedule(s.p)
        ids, k, v = s.tokens(at, 1)
        q = torch.randn(s.G, s.d, generator=T.gen(at)).to(T.DT[dtype])
        out = s.decode(q, ids, k, v, [at])
        assert flagged(s)
        s.ref_append(ids, k, v, [at])
        rest(s)
        s.check_out(out, q, [at])
        out = s.decode(q, None, None, None, [at])
        assert flagged(s)
        s.check_out(out, q, [at])
        at += 1


@pytest.mark.parametrize("n,H,Hkv", [(90, 5, 5), (700, 5, 5), (700, 8, 2), (13000, 2, 2)])
def test_rows_that_are_not_the_kept_positions_are_flagged(n, H, Hkv):
    """A count above or below the never-evicted positions of the keep codes: flagged by the coding,
    and the rows there are stay right."""
    pol = [4, 2, 0, 3, 1] if Hkv == H else [4, 4, 4, 4, 2, 2, 2, 2]
    s = T.Setup(51, L=1, H=H, Hkv=Hkv, n=n, policies=pol)
    rows = s.cache.rows.clone()
    s.compact()
    assert int(s.err.item()) == 0
    s.check()
    for c in range(s.gk):
        for by in (1, -1, 3000, -int(rows[c])):
            if by == 0 or int(rows[c]) + by < 0:
                continue
            s.cache.rows[c] += by
            s.compact()
            assert flagged(s), (c, by)
            s.cache.rows.copy_(rows)
    s.compact()
    assert int(s.err.item()) == 0
    s.check()


@pytest.mark.parametrize("m", [1, 8, 70, 0])
def test_a_pool_that_ran_out_goes_on_when_it_is_made_larger(m):
    """Calls that find no page leave the counter at the pool's end, however often they are made; a
    larger pool with the old pages in front serves from there on.  m = 0: decode steps."""
    s = T.Setup(52, B=2, L=2, H=3, n=64, policies=[4, 3, 4], max_new=400, pages=1)
    s.compact()
    at, room = 64, [r.rows for r in s.ref]
    for step in range(3):
        ids, k, v = s.tokens(step, max(m, 1))
        pos = [at + step * max(m, 1)] * 2
        if m:
            s.append(ids, k, v, pos)
        else:
            q = torch.randn(s.G, s.d, generator=T.gen(step)).to(T.DT[s.dtype])
            s.decode(q, ids, k, v, pos)
        assert fg.fastgen_read_error(s.err) == fg.FG_ECAPACITY
        assert int(s.cache.next_page.item()) == s.cache.c.n_pages
        room = s.cache.rows.cpu().tolist()
        s.ref_append(ids, k, v, pos, room=room)
    s.check()
    s.err.zero_()
    old, count = s.cache, s.cache.c.n_pages
    kept = [x.clone() for x in (old.k_pages, old.v_pages, old.exps, old.pos)]
    s.set_pages(count + 60)
    for x, y in zip((s.cache.k_pages, s.cache.v_pages, s.cache.exps, s.cache.pos), kept):
        x[:count] = y
    at += 3 * max(m, 1)
    for step in range(70 if m == 0 else 3):
        ids, k, v = s.tokens(10 + step, max(m, 1))
        pos = [at + step * max(m, 1)] * 2
        if m:
            s.append(ids, k, v, pos)
        else:
            q = torch.randn(s.G, s.d, generator=T.gen(step)).to(T.DT[s.dtype])
            s.decode(q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
    assert fg.fastgen_read_error(s.err) == fg.FG_OK
    gpu = s.check()
    taken = [x for c in range(s.gk) for r in (False, True) for x in gpu.pages(c, r) if x >= 0]
    assert sorted(taken) == list(range(int(s.cache.next_page.item())))  # each page once, none lost


@pytest.mark.parametrize("n", [60, 1300])
@pytest.mark.parametrize("captured", [False, True])
def test_a_step_sees_descriptors_that_the_launch_before_it_wrote(n, captured):
    """Policies copied into the descriptors on the device, right before each step, with nothing
    between: the step places its token by them."""
    steps = 24
    s = T.Setup(53, L=1, H=4, n=n, policies=[4], max_new=steps + 4)
    s.compact()
    desc = [s.cache.caches.clone(), s.cache.caches.clone()]
    desc[1][:, 0] = P.S
    ids, k, v = s.tokens(1, 1)
    ids[:] = 200  # neither special nor punctuation
    q = torch.randn(s.G, s.d, generator=T.gen(1)).to(torch.bfloat16)
    io = [T.dev(x) for x in (q, k, v, ids)]
    pos = [T.dev([n + i], torch.int32) for i in range(steps)]
    outs = torch.zeros(steps, s.G, s.d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fg.fastgen_decode_q8_workspace_bytes(s.p, s.cache), dtype=torch.uint8,
                     device="cuda")

    def run():
        for i in range(steps):
            s.cache.caches.copy_(desc[i % 2])
            fg.fastgen_decode_attn_q8(s.p, s.cache, *io, s.special, s.punct, pos[i], None, outs[i],
                                      ws, s.err)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graph.replay()
    else:
        run()
    torch.cuda.synchronize()
    for i in range(steps):
        if i % 2 == 0:
            s.ref_append(ids, k, v, [n + i])
        s.check_out(outs[i], q, [n + i])
    assert s.cache.rows.tolist() == [n + steps // 2] * s.gk and int(s.err.item()) == 0
