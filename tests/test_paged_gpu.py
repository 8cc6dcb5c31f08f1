"""The position rotation and the paged 8-bit caches on the GPU against plain
float64 statements (paged_ref.py): codes, exponents, positions, row counts and
page tables exactly where no rotation comes before the rounding, outputs
within bounds derived there."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref as P
from adaptive_head_kv_gb300 import fastgen as fg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODE = {"bf16": fg.FG_BF16, "fp32": fg.FG_FP32}
SPECIAL, PUNCT = [1, 7], [11, 402, 31999]


def dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).cuda().contiguous()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(x):
    return x.double().cpu().numpy()


# ---------------------------------------------------------------- rotation
def table(rot, base=10000.0):
    inv = base ** (-np.arange(0, rot, 2) / rot)
    return inv, dev(fg.fastgen_rope_table(inv))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,half", [(128, 128, False), (128, 128, True), (128, 64, True),
                                        (128, 48, False), (64, 64, True), (64, 32, False),
                                        (64, 16, True), (128, 112, True)])
@pytest.mark.parametrize("B,L,H,Hkv,n", [(1, 1, 1, 0, 1), (2, 3, 8, 2, 37), (1, 2, 24, 24, 130)])
def test_rope(dtype, d, rot, half, B, L, H, Hkv, n):
    p = fg.Params(B, L, H, n, d, CODE[dtype], 0.95, 0.3, 0.3, 0.0, Hkv)
    G, gk = B * L * H, B * L * (Hkv or H)
    g = gen(n + rot)
    Q, K = (torch.randn(x, n, d, generator=g).to(DT[dtype]) for x in (G, gk))
    pos = torch.randint(0, 1 << 30, (B, n), generator=g, dtype=torch.int32)
    inv, turns = table(rot)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    for at in (pos, None):
        Qd, Kd = dev(Q), dev(K)
        Qo, Ko = torch.empty_like(Qd), torch.empty_like(Kd)
        atd = None if at is None else dev(at)
        fg.fastgen_rope(p, Qd, Kd, atd, rope, Qo, Ko)
        where = np.broadcast_to(np.arange(n), (B, n)) if at is None else at.numpy()
        for x, y in ((Q, Qo), (K, Ko)):
            x64 = f64(x).reshape(B, -1, n, d)
            want = P.rotate(x64, where[:, None], inv, half)
            # two products, a sum, and (cos, sin) within 2^-22 each (an angle's fraction to 2^-25
            # half turns, a few roundings of 2^-24): 2^-21 of the pair's size.  A table entry is
            # inv_freq / 2 pi with 2^-52 relative error, times 2^30: 2^-22 turns at these positions
            size = np.abs(x64).reshape(B, -1, n, d)
            pair = size.max(-1, keepdims=True) * 2
            angle = 2.0 ** -19 if at is not None else 2.0 ** -21
            half_step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
            bound = pair * (2.0 ** -21 + angle) + half_step * np.abs(want)
            assert (np.abs(f64(y).reshape(want.shape) - want) <= bound).all()
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
        fg.fastgen_rope(p, Qd, Kd, atd, rope, Qd, Kd)  # in place
        assert torch.equal(Qd, Qo) and torch.equal(Kd, Ko)
        only = torch.empty_like(Ko)
        fg.fastgen_rope(p, None, dev(K), atd, rope, None, only)
        assert torch.equal(only, Ko)


# ------------------------------------------------------------- the caches
class Setup:
    """A prompt's paged caches through the library's plan, and the reference."""

    def __init__(self, seed, B=1, L=2, H=5, Hkv=0, n=150, d=128, dtype="bf16", r_l=0.3, max_new=40,
                 policies=None, pages=None, plant=None):
        g = gen(seed)
        self.p = fg.Params(B, L, H, n, d, CODE[dtype], 0.95, r_l, 0.3, 0.0, Hkv)
        self.B, self.n, self.d, self.dtype, self.max_new = B, n, d, dtype, max_new
        self.G, self.gk = B * L * H, B * L * (Hkv or H)
        self.R, self.hl = self.G // self.gk, L * (Hkv or H)
        self.w = int(np.ceil(float(np.float32(r_l)) * n))
        pol = torch.tensor([(policies or range(5))[i % len(policies or range(5))]
                            for i in range(self.G)], dtype=torch.int8)
        keep = torch.zeros(self.G, n, dtype=torch.uint8)
        frac = [0.02, 0.1, 0.3, 0.3, 1.0]
        for i in range(self.G):
            st = torch.rand(n, generator=g) < frac[int(pol[i])]
            if int(pol[i]) == P.S and i % 2:
                st[:] = False  # an empty cache
            keep[i, st] = 1
            if int(pol[i]) == P.SPFL and self.w:
                win = torch.arange(n) >= n - self.w
                keep[i, win & ~st] = 2
        self.policy, self.keep = pol, keep
        self.K, self.V = (torch.randn(self.gk, n, d, generator=g).to(DT[dtype]) for _ in range(2))
        self.K[..., 5] *= 6.0
        if plant:
            plant(self)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        tl = fg.fastgen_paged_table_len(self.p, max_new)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache = fg.PagedCache(self.p, None, None, None, None, torch.full((tl,), -7, **i32),
                                   torch.zeros(self.gk, 6, **i32), torch.zeros(self.gk, **i32),
                                   torch.zeros(1, **i32))
        self.info = fg.fastgen_paged_plan(self.p, dev(pol), dev(keep), max_new, self.cache)
        self.fill = 0x35  # a finite code: 0.8125
        self.set_pages(self.info.max_pages if pages is None else self.info.pages + pages)
        self.special, self.punct = dev(SPECIAL, torch.int32), dev(PUNCT, torch.int32)
        self.ref = []
        for c in range(self.gk):
            g0 = (c // (Hkv or H)) * H + (c % (Hkv or H)) * self.R
            st = (keep[g0: g0 + self.R] == 1).any(0)
            win = (keep[g0: g0 + self.R] == 2).any(0) & ~st
            policy = int(pol[g0: g0 + self.R].max())
            cap = (int(st.sum()) + max_new + 63) // 64 * 64 or 64
            r = P.RefCache(policy, self.w, cap, d)
            for side in (*r.seg.values(), *r.ring.values()):
                side.codes[:] = 0.8125
            r.compact(st.nonzero()[:, 0].tolist(), win.nonzero()[:, 0].tolist() if r.w else [],
                      f64(self.K[c]), f64(self.V[c]))
            self.ref.append(r)

    def set_pages(self, count):
        full = lambda shape, v, t: torch.full(shape, v, dtype=t, device="cuda")
        d = self.d
        self.cache.set_pages(full((count, 64, d), self.fill, torch.uint8),
                             full((count, 64, d), self.fill, torch.uint8),
                             full((count, 8), 17, torch.int8), full((count, 64), -3, torch.int32))

    def compact(self):
        fg.fastgen_compact_q8(self.p, dev(self.K), dev(self.V), dev(self.keep), self.cache, self.err)

    def tokens(self, seed, m):
        g = gen(seed)
        ids = torch.randint(100, 300, (self.B, m), generator=g, dtype=torch.int32)
        pick = torch.rand(self.B, m, generator=g)
        ids[pick < 0.2] = PUNCT[1]
        ids[pick > 0.9] = SPECIAL[1]
        k, v = (torch.randn(self.gk, m, self.d, generator=g) * torch.exp(
            1.5 * torch.randn(self.gk, m, 1, generator=g)) for _ in range(2))
        return ids, k.to(DT[self.dtype]), v.to(DT[self.dtype])

    def append(self, ids, k, v, pos, n_new=None, rope=None):
        m = ids.shape[1]
        ws = torch.empty(fg.fastgen_append_q8_workspace_bytes(self.p, m), dtype=torch.uint8,
                         device="cuda")
        fg.fastgen_append_q8(self.p, self.cache, dev(k), dev(v), dev(ids),
                             None if n_new is None else dev(n_new, torch.int32), self.special,
                             self.punct, dev(pos, torch.int32), rope, ws, self.err)

    def ref_append(self, ids, k, v, pos, n_new=None, turn=None, room=None):
        for c, r in enumerate(self.ref):
            b = c // self.hl
            cnt = ids.shape[1] if n_new is None else n_new[b]
            if pos[b] < 0 or cnt == 0:
                continue
            kinds = [(int(t) in SPECIAL, int(t) in PUNCT) for t in ids[b, :cnt]]
            kk = f64(k[c, :cnt])
            if turn:
                kk = turn(kk, pos[b] + np.arange(cnt))
            r.append(kk, f64(v[c, :cnt]), kinds, pos[b], None if room is None else room[c])

    def check(self, rotated=False, empty=True):
        """Every cache's rows against the reference.  rotated: keys that were rotated before
        their rounding may differ by what the rotation's rounding moves.  empty: ring slots
        that no row was ever put in are compared too."""
        gpu = P.GpuPages(self.cache)
        for c, r in enumerate(self.ref):
            assert gpu.rows[c] == r.rows, (c, gpu.rows[c], r.rows)
            assert list(gpu.caches[c][:2]) == [r.policy, r.w]
            for ring, side, count, pos in ((False, r.seg, r.rows, r.seg_pos[: r.rows]),
                                           (True, r.ring, r.w, r.ring_pos)):
                if count == 0:
                    continue
                got = gpu.segment(c, ring, count)
                assert np.array_equal(got["pos"], pos), (c, ring)
                for x in "kv":
                    assert np.array_equal(got["e" + x], side[x].e[: -(-count // 16)]), (c, ring, x)
                    want = side[x].codes[:count]
                    if not empty:
                        want = np.where((pos >= 0)[:, None], want, got[x])
                    if x == "k" and rotated:
                        # a value that the 32-bit rotation moves across a rounding border comes
                        # out one step away: 2^-3 of it (2^-9 among the subnormals); rare
                        off = got[x] != want
                        assert off.mean() <= 1e-3
                        assert (np.abs(got[x] - want) <= np.maximum(2.0 ** -3 * np.maximum(
                            np.abs(want), np.abs(got[x])), 2.0 ** -9)).all()
                    else:
                        assert np.array_equal(got[x], want, equal_nan=True), (c, ring, x)
                if rotated:  # later steps start from what is stored
                    side["k"].codes[:count] = got["k"]
        return gpu

    def decode(self, q, ids, k, v, pos, rope=None, out=None, reuse=None):
        ws = reuse
        if ws is None:
            ws = torch.full((fg.fastgen_decode_q8_workspace_bytes(self.p, self.cache),), 0xFF,
                            dtype=torch.uint8, device="cuda")
        if out is None:
            out = torch.full((self.G, self.d), 3.5, dtype=DT[self.dtype], device="cuda")
        new = [None if x is None else dev(x) for x in (k, v, ids)]
        fg.fastgen_decode_attn_q8(self.p, self.cache, dev(q), new[0], new[1], new[2], self.special,
                                  self.punct, dev(pos, torch.int32), rope, out, ws, self.err)
        return out

    def check_out(self, out, q, pos, turn=None, idle=3.5):
        got = f64(out)
        for g in range(self.G):
            hkv = self.p.Hkv or self.p.H
            c = (g // self.p.H) * hkv + (g % self.p.H) // self.R
            b = c // self.hl
            if pos[b] < 0:
                assert (got[g] == idle).all()
                continue
            qq = f64(q[g])
            if turn:
                qq = turn(qq, pos[b])
            k, v, ev = self.ref[c].kv(pos[b])
            want, weight, products, floor = P.attend(qq, k, v, ev, 1 / np.sqrt(self.d))
            bound = P.decode_bound(want, weight, products, floor, self.dtype)
            assert (np.abs(got[g] - want) <= bound).all(), (
                g, np.abs(got[g] - want).max(), bound.min(), len(k))


SHAPES = [
    dict(),
    dict(d=64, n=77, dtype="fp32"),
    dict(H=8, Hkv=2, n=333, d=128),
    dict(H=8, Hkv=4, n=65, d=64, B=2),
    dict(H=8, Hkv=1, L=3, n=200, d=128, dtype="fp32"),
    dict(n=1, L=1),
    dict(n=64, r_l=0.01),
    dict(n=129, r_l=0.0),
    dict(n=40, r_l=1.0, d=64),
    dict(n=1300, L=1, r_l=0.45),
]


@pytest.mark.parametrize("kw", SHAPES)
def test_plan_and_compact(kw):
    s = Setup(1, **kw)
    s.compact()
    gpu = s.check()
    assert int(s.err.item()) == 0
    # the plan: pages in order, each once, -1 where a cache may grow, counts as documented
    used, now, most, entries = [], 0, 0, 0
    for c, r in enumerate(s.ref):
        seg, ring = gpu.pages(c, False), gpu.pages(c, True)
        have = -(-r.rows // 64)
        assert len(seg) == max(1, -(-(r.rows + s.max_new) // 64)) and len(ring) == -(-r.w // 64)
        assert (seg[have:] == -1).all()
        used += list(seg[:have]) + list(ring)
        now, most, entries = now + have + len(ring), most + len(seg) + len(ring), entries + len(seg) + len(ring)
    assert used == list(range(now))
    assert (s.info.pages, s.info.max_pages, s.info.table_used) == (now, most, entries)
    assert int(s.cache.next_page.item()) == now
    # what no row needs stays as it was
    for c, r in enumerate(s.ref):
        for ring, count in ((False, r.rows), (True, r.w)):
            pg = gpu.pages(c, ring)
            pg = pg[pg >= 0]
            assert (gpu.pos[pg].reshape(-1)[count:] == -3).all()
            assert (gpu.codes["k"][pg].reshape(-1, s.d)[count:] == 0.8125).all()
            assert (gpu.e[pg].reshape(-1, 2)[-(-count // 16):] == 17).all()
    rest = np.setdiff1d(np.arange(s.cache.c.n_pages), used)
    assert (gpu.pos[rest] == -3).all() and (gpu.codes["v"][rest] == 0.8125).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_compact_special_values(dtype):
    """Zero, tiny, huge, infinite and NaN values; borders of the exponent rule."""
    def plant(s):
        big = torch.finfo(DT[dtype]).max
        for c in range(s.gk):
            s.K[c, 0:16] = 0.0
            s.K[c, 16:32] = 2.0 ** -120
            s.K[c, 32] = big
            s.V[c, 3, 7], s.V[c, 4, 8], s.V[c, 5, 9] = float("inf"), float("-inf"), float("nan")
            s.V[c, 40:56] = 0.0
            s.V[c, 41, 0] = 448.0 * 2.0 ** 3
            s.V[c, 60, :] = 449.9 if dtype == "fp32" else 450.0
            s.V[c, 70, :] = 2.0 ** -9 * torch.arange(s.d)
            s.V[c, 71, 0] = 448.0
    s = Setup(2, L=1, H=4, n=96, dtype=dtype, policies=[4, 4, 3, 2], plant=plant)
    s.compact()
    s.check()
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("kw", SHAPES)
@pytest.mark.parametrize("m", [1, 2, 17, 40])
def test_append(kw, m):
    s = Setup(3, max_new=100, **kw)
    s.compact()
    for step in range(2):
        ids, k, v = s.tokens(10 * m + step, m)
        pos = [s.n + step * m + 5 * b for b in range(s.B)]
        n_new = [max(0, m - 3 * b) for b in range(s.B)]
        s.append(ids, k, v, pos, n_new)
        s.ref_append(ids, k, v, pos, n_new)
        gpu = s.check()
    assert int(s.err.item()) == 0
    taken = [x for c in range(s.gk) for r in (False, True) for x in gpu.pages(c, r) if x >= 0]
    assert sorted(taken) == list(range(int(s.cache.next_page.item())))  # each page once


def test_append_longer_than_the_window_and_ragged():
    s = Setup(4, B=3, L=1, n=50, max_new=700, r_l=0.4)
    s.compact()
    ids, k, v = s.tokens(5, 601)
    pos, n_new = [50, -1, 60], [601, 600, 0]
    s.append(ids, k, v, pos, n_new)
    s.ref_append(ids, k, v, pos, n_new)
    s.check()
    ids, k, v = s.tokens(6, 9)
    s.append(ids, k, v, [651, 50, 61])
    s.ref_append(ids, k, v, [651, 50, 61])
    s.check()
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d,rot,dtype", [(128, 128, "bf16"), (64, 64, "fp32"), (128, 48, "fp32"),
                                         (64, 16, "bf16")])
def test_append_and_decode_rotate(half, d, rot, dtype):
    inv, turns = table(rot)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    turn = lambda x, at: P.rotate(x, at, inv, half)
    s = Setup(7, B=2, H=4, Hkv=2, d=d, dtype=dtype, n=70, max_new=64)
    s.compact()
    ids, k, v = s.tokens(1, 20)
    pos = [70, 100000]
    s.append(ids, k, v, pos, rope=rope)
    s.ref_append(ids, k, v, pos, turn=turn)
    s.check(rotated=True)
    pos = [90, 100020]
    ids, k, v = s.tokens(2, 1)
    q = torch.randn(s.G, d, generator=gen(3)).to(DT[dtype])
    out = s.decode(q, ids, k, v, pos, rope)
    s.ref_append(ids, k, v, pos, turn=turn)
    s.check(rotated=True)
    s.check_out(out, q, pos, turn)
    assert int(s.err.item()) == 0


def test_rows_out_leaves_rows_and_the_call_repeats():
    s = Setup(8, n=90, max_new=64)
    s.compact()
    before = s.cache.rows.clone()
    s.cache.rows_out = torch.zeros_like(before)
    s.cache.c.rows_out = s.cache.rows_out.data_ptr()
    ids, k, v = s.tokens(1, 33)
    for _ in range(2):
        s.append(ids, k, v, [90])
        assert torch.equal(s.cache.rows, before)
    s.ref_append(ids, k, v, [90])
    s.check()


def test_capacity():
    """The pool, then a table, runs out: flagged, what fits is stored, nothing else touched."""
    s = Setup(9, L=1, H=2, n=60, policies=[4, 4], max_new=200, pages=1)
    s.compact()
    ids, k, v = s.tokens(1, 70)  # both caches want rows 60 .. 129: 2 more pages each
    s.append(ids, k, v, [60])
    assert fg.fastgen_read_error(s.err) == fg.FG_ECAPACITY
    rows = s.cache.rows.cpu().tolist()
    assert sorted(rows) == [64, 128]  # one cache got the one free page
    s.ref_append(ids, k, v, [60], room=rows)
    s.check()
    s.err.zero_()
    s = Setup(9, L=1, H=2, n=60, policies=[4, 3], max_new=4)
    s.compact()
    ids, k, v = s.tokens(1, 1)
    for t in range(60, 66):
        q = torch.randn(s.G, s.d, generator=gen(t)).to(DT[s.dtype])
        out = s.decode(q, ids, k, v, [t])
        s.ref_append(ids, k, v, [t])
        s.check()
        s.check_out(out, q, [t])
        assert fg.fastgen_read_error(s.err) == (fg.FG_OK if t < 64 else fg.FG_ECAPACITY)


@pytest.mark.parametrize("kw", SHAPES + [dict(H=4, Hkv=2, n=700, L=1), dict(n=2600, L=1, H=4, Hkv=1)])
def test_decode_steps(kw):
    steps = 6 if kw.get("n", 0) > 1000 else 40
    s = Setup(11, max_new=steps, pages=None, **kw)
    s.compact()
    for st in range(steps):
        ids, k, v = s.tokens(100 + st, 1)
        pos = [s.n + st + 2 * b if st % 5 or b == 0 else -1 for b in range(s.B)]
        q = (torch.randn(s.G, s.d, generator=gen(st)) * (1 + st % 3)).to(DT[s.dtype])
        out = s.decode(q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
        if st % 6 == 0 or st == steps - 1:
            s.check()
        s.check_out(out, q, pos)
    assert int(s.err.item()) == 0


def test_decode_without_a_new_token_and_empty_caches():
    s = Setup(12, L=2, H=4, n=100, policies=[0, 4, 3, 0])
    s.compact()
    q = torch.randn(s.G, s.d, generator=gen(1)).to(DT[s.dtype])
    out = s.decode(q, None, None, None, [99])
    s.check()
    s.check_out(out, q, [99])
    empty = [g for g in range(s.G) if s.ref[g].rows == 0 and s.ref[g].w == 0]
    assert empty and (out[empty] == 0).all()
    # the window slides away when time goes on without rows
    out = s.decode(q, None, None, None, [99 + s.w - 1])
    s.check_out(out, q, [99 + s.w - 1])
    out = s.decode(q, None, None, None, [5000])
    s.check_out(out, q, [5000])


def test_nan_outside_the_cache_and_inside_it():
    """Rows that are not in the cache may hold NaN; a NaN inside it stays with its heads."""
    s = Setup(13, L=1, H=5, n=100)
    s.fill = 0x7F  # NaN
    s.set_pages(s.info.max_pages)
    s.compact()
    q = torch.randn(s.G, s.d, generator=gen(1)).to(DT[s.dtype])
    out = s.decode(q, None, None, None, [99])
    s.check_out(out, q, [99])
    gpu = P.GpuPages(s.cache)
    page = int(gpu.pages(4, False)[0])  # the full cache
    s.cache.k_pages[page, 3, 5] = 0x7F
    out = s.decode(q, None, None, None, [99])
    assert torch.isnan(out[4]).all() and torch.isfinite(out[:4]).all()


def test_large_exponents_of_values_and_keys():
    """Blocks of very different sizes: V's exponent rides on the weight, K's on the score."""
    def plant(s):
        s.V[:, ::31] *= 2.0 ** 60
        s.V[:, 1::31] *= 2.0 ** -60
        s.K[:, 2::37] *= 2.0 ** -40
        s.K[:, 50] *= 30.0
    for dtype in ("bf16", "fp32"):
        s = Setup(14, L=1, H=8, Hkv=4, n=210, dtype=dtype, policies=[4, 4, 3, 3, 2], plant=plant)
        s.compact()
        s.check()
        q = torch.randn(s.G, s.d, generator=gen(1)).to(DT[dtype])
        for scale in (1.0, 2.0 ** -30, 2.0 ** 5):
            qs = (q.float() * scale).to(DT[dtype])
            out = s.decode(qs, None, None, None, [209])
            s.check_out(out, qs, [209])


def test_bad_pages_and_counts_are_flagged_not_followed():
    s = Setup(15, L=1, H=5, n=200)
    s.compact()
    ids, k, v = s.tokens(1, 3)
    q = torch.randn(s.G, s.d, generator=gen(1)).to(DT[s.dtype])
    table, caches, rows = s.cache.page_table, s.cache.caches, s.cache.rows
    keep = [x.clone() for x in (table, caches, rows)]

    def restore():
        for x, y in zip((table, caches, rows), keep):
            x.copy_(y)
        s.err.zero_()

    full = P.GpuPages(s.cache).caches[4]
    for bad in (s.cache.c.n_pages, 1 << 30, -5):
        table[int(full[2]) + 1] = bad
        out = s.decode(q, None, None, None, [199])
        assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
        assert torch.isfinite(out).all()
        s.append(ids, k, v, [200])
        s.compact()
        assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
        restore()
    for col, bad in ((2, -1), (2, 1 << 30), (4, 1 << 30), (3, 0)):
        caches[3:, col] = bad
        out = s.decode(q, ids[:, :1], k[:, :1], v[:, :1], [200])
        s.append(ids, k, v, [201])
        s.compact()
        assert fg.fastgen_read_error(s.err) in (fg.FG_EINVAL, fg.FG_ECAPACITY)
        assert torch.isfinite(out).all()
        restore()
    for bad in (1 << 30, -9):
        rows[4] = bad
        s.decode(q, None, None, None, [199])
        assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
        restore()


def test_reschedule_and_other_stream_and_graph():
    """A captured step replayed with the positions moving on the device gives the steps' results;
    the work list may be rebuilt; a stream of its own."""
    steps = 30
    a, b = (Setup(16, B=2, L=1, H=4, Hkv=2, n=600, max_new=steps) for _ in range(2))
    side = torch.cuda.Stream()
    ids, k, v = zip(*(a.tokens(50 + i, 1) for i in range(steps)))
    q = [torch.randn(a.G, a.d, generator=gen(i)).to(torch.bfloat16) for i in range(steps)]
    a.compact()
    want = []
    for i in range(steps):
        if i == 10:
            a.cache.schedule(a.p)
        want.append(a.decode(q[i], ids[i], k[i], v[i], [600 + i, 700 + i]).clone())
    b.compact()
    torch.cuda.synchronize()
    qd, kd, vd, idd = dev(q[0]), dev(k[0]), dev(v[0]), dev(ids[0])
    pos = dev([600, 700], torch.int32)
    out = torch.zeros(b.G, b.d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fg.fastgen_decode_q8_workspace_bytes(b.p, b.cache), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            fg.fastgen_decode_attn_q8(b.p, b.cache, qd, kd, vd, idd, b.special, b.punct, pos, None,
                                      out, ws, b.err)
            pos += 1
        for i in range(steps):
            for x, y in ((qd, q[i]), (kd, k[i].reshape(kd.shape)), (vd, v[i].reshape(vd.shape)),
                         (idd, ids[i])):
                x.copy_(y)
            graph.replay()
            got = out.clone()
            side.synchronize()
            if i < 10:  # the same work list: the same bits
                assert torch.equal(got, want[i])
            b.ref_append(ids[i], k[i], v[i], [600 + i, 700 + i])
            b.check_out(got, q[i], [600 + i, 700 + i])
    assert pos.tolist() == [630, 730]


def test_calls_are_bitwise_repeatable():
    outs = []
    for _ in range(3):
        s = Setup(17, L=3, H=8, Hkv=8, n=400, max_new=64)
        s.compact()
        ids, k, v = s.tokens(1, 40)
        s.append(ids, k, v, [400])
        q = torch.randn(s.G, s.d, generator=gen(2)).to(torch.bfloat16)
        outs.append(s.decode(q, ids[:, :1], k[:, :1], v[:, :1], [440]))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------ the whole path
@pytest.mark.parametrize("dtype,H,Hkv,d,half", [("bf16", 8, 8, 128, False), ("bf16", 8, 2, 64, True),
                                                ("fp32", 4, 2, 128, True)])
def test_session_from_projections_to_steps(dtype, H, Hkv, d, half):
    """PagedSession on queries and keys as projected: rotation, profile, plan, coding, a turn of
    several tokens, steps (eager and captured); the caches against the reference built from the
    profile's own keep codes, and the 16-bit session's outputs nearby."""
    from adaptive_head_kv_gb300.session import FastGenSession, PagedSession, make_params

    B, L, n, steps, turn_len = 2, 2, 210, 6, 9
    rot = d if not half else d // 2
    inv, turns = table(rot)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    turn = lambda x, at: P.rotate(x, at, inv, half)
    p = make_params(B, L, H, n, d, dtype, 0.9, 0.3, 0.3, Hkv=Hkv)
    G, gk = B * L * H, B * L * Hkv
    g = gen(3)
    total = n + turn_len + 2 * steps
    Q, K, V = (torch.randn(x, total, d, generator=g) for x in (G, gk, gk))
    Q, K, V = (x.to(DT[dtype]) for x in (Q, K, V))
    ids = torch.randint(100, 300, (B, total), generator=g, dtype=torch.int32)
    ids[torch.rand(B, total, generator=g) < 0.1] = PUNCT[1]
    ids[:, 0] = SPECIAL[0]
    s = PagedSession(p, SPECIAL, PUNCT, turn_len + 2 * steps, guard=True, rope=rope)
    Qp, Kp, Vp = (dev(x[:, :n]) for x in (Q, K, V))
    saved = torch.arange(G, dtype=torch.int8) // (H // Hkv) % 5  # every entry of the shortlist
    s.prefill_with_policy(Qp, Kp, Vp, dev(ids[:, :n]), saved)
    assert torch.equal(Qp.cpu(), Q[:, :n])  # the caller's tensors stay
    # the reference's caches, from the rotated keys that were profiled
    Kr = f64(s._rotated[1])
    keep, pol = s.keep.cpu(), s.policy.cpu()
    R, hl = G // gk, L * Hkv
    w = int(np.ceil(float(np.float32(0.3)) * n))
    ref = []
    for c in range(gk):
        g0 = (c // Hkv) * H + (c % Hkv) * R
        st = (keep[g0: g0 + R] == 1).any(0)
        win = (keep[g0: g0 + R] == 2).any(0) & ~st
        r = P.RefCache(int(pol[g0: g0 + R].max()), w, 1024, d)
        r.compact(st.nonzero()[:, 0].tolist(), win.nonzero()[:, 0].tolist(), Kr[c], f64(Vp[c]))
        ref.append(r)
    assert set(r.policy for r in ref) == set(range(5))
    h = Setup.__new__(Setup)  # its comparisons, on this session's cache
    h.p, h.cache, h.ref, h.G, h.gk, h.R, h.hl, h.d, h.dtype = (
        s.p, s.cache, ref, G, gk, R, hl, d, dtype)
    h.check(empty=False)
    s.append(dev(K[:, n: n + turn_len]), dev(V[:, n: n + turn_len]), dev(ids[:, n: n + turn_len]), n)
    h.ref_append(ids[:, n: n + turn_len], K[:, n: n + turn_len], V[:, n: n + turn_len], [n] * B,
                 turn=turn)
    h.check(rotated=True, empty=False)
    s.reschedule()
    # the 16-bit session on rotated inputs, token by token
    plain = FastGenSession(p, SPECIAL, PUNCT, turn_len + 2 * steps)
    every = torch.arange(total, dtype=torch.int32).expand(B, total)
    pt = make_params(B, L, H, total, d, dtype, 0.9, 0.3, 0.3, Hkv=Hkv)
    Qa, Ka = torch.empty_like(dev(Q)), torch.empty_like(dev(K))
    fg.fastgen_rope(pt, dev(Q), dev(K), dev(every), rope, Qa, Ka)
    plain.prefill_with_policy(*(x[:, :n].contiguous() for x in (Qa, Ka, dev(V))),
                              dev(ids[:, :n]), saved)
    assert torch.equal(plain.keep, s.keep)
    outs = {}
    for t in range(n, total):
        outs[t] = plain.decode(Qa[:, t].contiguous(), Ka[:, t].contiguous(), dev(V[:, t]),
                               dev(ids[:, t]), t).clone()
    at = n + turn_len
    for t in range(at, at + steps):
        out = s.decode(dev(Q[:, t]), dev(K[:, t]), dev(V[:, t]), dev(ids[:, t]), t)
        h.ref_append(ids[:, t: t + 1], K[:, t: t + 1], V[:, t: t + 1], [t] * B, turn=turn)
        h.check(rotated=True, empty=False)
        h.check_out(out, Q[:, t], [t] * B, turn)
        rms = outs[t].float().pow(2).mean().sqrt()
        assert (out.float() - outs[t].float()).pow(2).mean().sqrt() < 0.1 * rms
    at += steps
    stack = lambda x: dev(x[:, at: at + steps].transpose(0, 1))
    pool = [x.clone() for x in (s.cache.k_pages, s.cache.v_pages, s.cache.exps, s.cache.pos,
                                s.cache.page_table, s.cache.rows, s.cache.next_page)]
    graph, gouts = s.capture_decode(stack(Q), stack(K), stack(V), stack(ids), at)
    graph.replay()
    torch.cuda.synchronize()
    captured = gouts.clone()
    for x, y in zip((s.cache.k_pages, s.cache.v_pages, s.cache.exps, s.cache.pos,
                     s.cache.page_table, s.cache.rows, s.cache.next_page), pool):
        x.copy_(y)
    for i in range(steps):
        t = at + i
        out = s.decode(dev(Q[:, t]), dev(K[:, t]), dev(V[:, t]), dev(ids[:, t]), t)
        assert torch.equal(out, captured[i])
        h.ref_append(ids[:, t: t + 1], K[:, t: t + 1], V[:, t: t + 1], [t] * B, turn=turn)
        h.check(rotated=True, empty=False)
        h.check_out(out, Q[:, t], [t] * B, turn)
    assert fg.fastgen_read_error(s.dev_err) == fg.FG_OK
    assert s.check_guards() == 0


# --------------------------------------------------------- calls less usual
@pytest.mark.parametrize("kw", [dict(B=2, L=16, H=32, n=70), dict(B=3, L=14, H=32, Hkv=32, n=33, d=64),
                                dict(B=4, L=16, H=32, Hkv=16, n=20, dtype="fp32")])
def test_many_caches_share_thread_blocks(kw):
    """More items than thread blocks: a block takes several caches, and parts of them."""
    s = Setup(20, max_new=8, **kw)
    assert s.cache.c.n_ctas < s.cache.c.n_work or s.gk < 900
    s.compact()
    for st in range(3):
        ids, k, v = s.tokens(st, 1)
        pos = [s.n + st if b != 1 else -1 for b in range(s.B)]
        q = torch.randn(s.G, s.d, generator=gen(st)).to(DT[s.dtype])
        out = s.decode(q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
        s.check_out(out, q, pos)
    s.check()
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("kw,idle", [
    (dict(B=4, L=4, H=8, n=2600, d=64, policies=[4, 4, 3, 4]), [[0], [3], [1, 2], [0, 1, 2], []]),
    (dict(B=40, L=3, H=8, n=70), [[0, 5, 31, 32, 39], range(1, 40), range(39), [7], range(40)]),
    (dict(B=3, L=10, H=64, Hkv=32, n=50, dtype="fp32"), [[1], [0, 2]]),
    (dict(B=2, L=2, H=64, Hkv=32, n=4200, policies=[4, 3, 1, 2]), [[0], [1]]),
    # every cache as long, lengths that end where caches do: no room for more items
    (dict(B=2, L=2, H=64, Hkv=16, n=4200, policies=[4, 3, 4, 1]), [[0], [1]]),
])
def test_idle_sequences_of_a_large_step(kw, idle):
    """The list is cut again for the sequences that take part, whichever they are."""
    s = Setup(28, max_new=8, **kw)
    assert int(s.cache.sched.view(torch.int32)[64 + 3]) > 0  # a list of equal lengths
    s.compact()
    now = np.full(s.B, s.n)
    for st, off in enumerate(idle):
        ids, k, v = s.tokens(st, 1)
        pos = [-1 if b in off else int(now[b]) for b in range(s.B)]
        q = torch.randn(s.G, s.d, generator=gen(st)).to(DT[s.dtype])
        out = s.decode(q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
        s.check_out(out, q, pos)
        now += [p >= 0 for p in pos]
    s.check()
    assert int(s.err.item()) == 0


def test_long_items_and_a_schedule_from_before_the_growth():
    """The last item of a segment takes thousands of later rows; then the list is made anew."""
    s = Setup(21, L=1, H=8, Hkv=2, n=30, policies=[4, 4, 4, 4, 3, 3, 1, 0], max_new=5000, r_l=0.9)
    s.compact()
    at = 30
    for m in (2500, 33, 32, 1):
        ids, k, v = s.tokens(m, m)
        s.append(ids, k, v, [at])
        s.ref_append(ids, k, v, [at])
        at += m
    s.check()
    q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
    old = s.decode(q, None, None, None, [at - 1])
    s.check_out(old, q, [at - 1])
    s.cache.schedule(s.p)
    assert s.cache.c.n_work > 2
    s.check_out(s.decode(q, None, None, None, [at - 1]), q, [at - 1])
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("m", [1, 7, 40])
def test_id_sets_none_empty_and_longer_than_a_warp(m):
    many = torch.arange(5000, 5070, dtype=torch.int32)
    for special, punct in ((None, None), (many, many + 1000), (many[:0], many[:33])):
        s = Setup(22, L=1, H=5, n=60, max_new=100)
        s.special, s.punct = (None if x is None else x.cuda() for x in (special, punct))
        s.compact()
        ids, k, v = s.tokens(3, m)
        ids[:, ::2] = 5000 + 69 if special is not None and len(special) else 5032
        ids[:, 1::5] = 6069
        real = (SPECIAL[:], PUNCT[:])
        SPECIAL[:], PUNCT[:] = ([] if x is None else x.tolist() for x in (special, punct))
        try:
            s.append(ids, k, v, [60])
            s.ref_append(ids, k, v, [60])
            s.check()
            q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
            out = s.decode(q, ids[:, :1], k[:, :1], v[:, :1], [60 + m])
            s.ref_append(ids[:, :1], k[:, :1], v[:, :1], [60 + m])
            s.check()
            s.check_out(out, q, [60 + m])
        finally:
            SPECIAL[:], PUNCT[:] = real


def test_nothing_to_do():
    """Idle batches and counts of zero leave everything as it was."""
    s = Setup(23, B=2, L=1, H=3, n=50)
    s.compact()
    before = [x.clone() for x in (s.cache.k_pages, s.cache.v_pages, s.cache.exps, s.cache.pos,
                                  s.cache.page_table, s.cache.rows, s.cache.next_page)]
    for m in (3, 40):
        ids, k, v = s.tokens(1, m)
        s.append(ids, k, v, [50, 50], [0, 0])
        s.append(ids, k, v, [-1, -7])
    q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
    out = s.decode(q, ids[:, :1], k[:, :1], v[:, :1], [-1, -1])
    assert (out == 3.5).all()
    for x, y in zip(before, (s.cache.k_pages, s.cache.v_pages, s.cache.exps, s.cache.pos,
                             s.cache.page_table, s.cache.rows, s.cache.next_page)):
        assert torch.equal(x, y)
    assert int(s.err.item()) == 0


def test_graphs_that_share_a_workspace_and_take_pages():
    """Two captured steps of two caches, one workspace, replayed in turn while the caches grow
    into pages not taken at capture."""
    a, b = (Setup(x, L=1, H=4, n=60, policies=[4, 3, 4, 1], max_new=80) for x in (24, 25))
    ws = torch.empty(max(fg.fastgen_decode_q8_workspace_bytes(x.p, x.cache) for x in (a, b)),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for s in (a, b):
        s.compact()
        ids, k, v = s.tokens(1, 1)
        q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
        io = [dev(x) for x in (q, k, v, ids)] + [dev([60], torch.int32),
                                                 torch.zeros(s.G, s.d, dtype=torch.bfloat16,
                                                             device="cuda")]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fg.fastgen_decode_attn_q8(s.p, s.cache, io[0], io[1], io[2], io[3], s.special, s.punct,
                                      io[4], None, io[5], ws, s.err)
            io[4] += 1
        graphs.append((s, g, io, (ids, k, v, q)))
    for st in range(70):
        for s, g, io, (ids, k, v, q) in graphs:
            g.replay()
            s.ref_append(ids, k, v, [60 + st])
            if st % 23 == 0 or st == 69:
                s.check_out(io[5], q, [60 + st])
    for s in (a, b):
        s.check()
        assert int(s.err.item()) == 0


def test_a_captured_append_outlives_a_longer_one():
    """The session's workspace grows with a longer call; the captured call keeps its own."""
    from adaptive_head_kv_gb300.session import PagedSession, make_params

    B, L, H, n, d, m = 2, 2, 4, 90, 64, 20
    p = make_params(B, L, H, n, d, "bf16", 0.9, 0.3, 0.3)
    rope = fg.Rope(table(d)[1])
    g, gk = gen(30), B * L * H
    prompt = [dev(torch.randn(gk, n, d, generator=g).to(torch.bfloat16)) for _ in range(3)]
    ids = dev(torch.randint(100, 300, (B, n), generator=g, dtype=torch.int32))
    turns = []
    for k in (m, 300, m):
        turns.append([dev(torch.randn(gk, k, d, generator=g).to(torch.bfloat16)) for _ in range(2)]
                     + [dev(torch.randint(100, 300, (B, k), generator=g, dtype=torch.int32))])
    at = [n, n + m, n + m + 300]
    a, b = (PagedSession(p, SPECIAL, PUNCT, 400, rope=rope) for _ in range(2))
    for s in (a, b):
        s.prefill_with_policy(*prompt, ids, torch.arange(gk, dtype=torch.int8) % 5)
    for x, t in zip(turns, at):
        a.append(*x, t)
    held, pos = [x.clone() for x in turns[0]], dev([n] * B, torch.int32)
    b.append(*held, dev([-1] * B, torch.int32))  # no sequence: sizes the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.append(*held, pos)
    graph.replay()
    b.append(*turns[1], at[1])
    other = torch.full((1 << 20,), 0xA5, dtype=torch.uint8, device="cuda")  # takes what was freed
    for x, y in zip(held, turns[2]):
        x.copy_(y)
    pos.fill_(at[2])
    graph.replay()
    torch.cuda.synchronize()
    assert (other == 0xA5).all()
    assert torch.equal(a.cache.rows, b.cache.rows) and int(a.dev_err) == 0 == int(b.dev_err)
    x, y = P.GpuPages(a.cache), P.GpuPages(b.cache)
    for c in range(gk):
        for ring, count in ((False, int(x.rows[c])), (True, int(x.caches[c][1]))):
            if count == 0:
                continue
            u, v = x.segment(c, ring, count), y.segment(c, ring, count)
            for key in u:
                assert np.array_equal(u[key], v[key], equal_nan=True), (c, ring, key)


def test_a_step_captured_before_the_list_was_made_anew_is_flagged():
    """Its thread blocks would not be the new list's: nothing is done, and the error word says so."""
    s = Setup(29, L=1, H=8, Hkv=2, n=30, policies=[4], max_new=1500)
    s.compact()
    q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
    qd, pos = dev(q), dev([29], torch.int32)
    out = torch.zeros(s.G, s.d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fg.fastgen_decode_q8_workspace_bytes(s.p, s.cache), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.fastgen_decode_attn_q8(s.p, s.cache, qd, None, None, None, s.special, s.punct, pos, None,
                                  out, ws, s.err)
    graph.replay()
    s.check_out(out, q, [29])
    ids, k, v = s.tokens(1, 1400)
    s.append(ids, k, v, [30])
    s.ref_append(ids, k, v, [30])
    pos.fill_(1429)
    graph.replay()  # the old list: its last items take the later rows
    s.check_out(out, q, [1429])
    before = s.cache.c.n_work
    s.cache.schedule(s.p)
    assert s.cache.c.n_work != before
    out.fill_(3.5)
    graph.replay()
    assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
    assert (out == 3.5).all()
    s.err.zero_()
    s.check_out(s.decode(q, None, None, None, [1429]), q, [1429])
    assert fg.fastgen_read_error(s.err) == fg.FG_OK


def test_a_list_of_another_cache_is_flagged():
    """A work list that does not belong to the cache: refused or flagged, never followed."""
    s = Setup(26, L=1, H=4, n=90)
    s.compact()
    torch.cuda.synchronize()
    s.cache.sched.view(torch.int32)[64 + 16:].fill_(1 << 28)
    q = torch.randn(s.G, s.d, generator=gen(1)).to(torch.bfloat16)
    s.decode(q, None, None, None, [89])
    assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
    s.err.zero_()
    s.cache.schedule(s.p)
    s.check_out(s.decode(q, None, None, None, [89]), q, [89])
    # descriptors that claim the same table over and over need more items than there can be
    s.cache.caches[:, 2] = 0
    s.cache.caches[:, 3] = 1 << 20
    s.cache.rows.fill_(1 << 26)
    for _ in range(2):
        try:
            s.cache.schedule(s.p)
        except fg.FastGenError as e:
            assert e.status == fg.FG_EINVAL
    # a ring larger than the window of the parameters
    t = Setup(27, L=1, H=4, n=90)
    t.cache.caches[3, 1] = 91
    t.compact()
    assert fg.fastgen_read_error(t.err) == fg.FG_EINVAL


@pytest.mark.parametrize("own_stream", [False, True])
def test_session_from_host_buffers_small_pool_and_stream(own_stream):
    """prefill_host rotates as prefill does; a pool without room to grow reports its capacity."""
    from adaptive_head_kv_gb300.session import PagedSession, make_params

    B, L, H, n, d = 1, 2, 4, 100, 64
    p = make_params(B, L, H, n, d, "bf16", 0.95, 0.3, 0.3)
    rope = fg.Rope.make(d, 10000.0, fg.FG_ROPE_HALF)
    stream = torch.cuda.Stream() if own_stream else None
    g = gen(1)
    Q, K, V = (torch.randn(L * H, n, d, generator=g).to(torch.bfloat16) for _ in range(3))
    ids = torch.randint(100, 200, (B, n), generator=g, dtype=torch.int32)
    sessions = []
    for host in (False, True):
        s = PagedSession(p, SPECIAL, PUNCT, 100, rope=rope, pages=0,
                         stream=None if host else stream)
        torch.cuda.synchronize()
        if host:
            h = [x.pin_memory() for x in (Q, K, V, ids)]
            s.prefill_host(*h, *(torch.empty_like(x, device="cuda") for x in h))
        else:
            s.prefill(dev(Q), dev(K), dev(V), dev(ids))
        torch.cuda.synchronize()
        sessions.append(s)
    a, b = sessions
    assert torch.equal(a.policy, b.policy) and torch.equal(a.keep, b.keep)
    assert a.cache.c.n_pages == a.info.pages
    pa, pb = P.GpuPages(a.cache), P.GpuPages(b.cache)
    for c in range(L * H):
        x, y = (z.segment(c, False, int(z.rows[c])) for z in (pa, pb))
        for key in x:
            assert np.array_equal(x[key], y[key])
    one = lambda: dev(torch.randn(L * H, d, generator=g).to(torch.bfloat16))
    tok = dev([[150]], torch.int32)
    assert [x.policy for x in a.descriptors()] == a.policy.cpu().tolist()
    full = any(x.policy == 4 for x in a.descriptors())
    for t in range(n, n + 64):
        torch.cuda.synchronize()
        a.decode(one(), one(), one(), tok, t)
    torch.cuda.synchronize()
    want = fg.FG_ECAPACITY if full else fg.FG_OK
    assert fg.fastgen_read_error(a.dev_err) == want
