"""Steps behind a shared prompt, the rows' weights, the cut to a budget and empty caches on the GPU
against plain float64 statements (paged_ref.py): what is stored exactly, outputs and weights within
bounds derived there and here."""
import numpy as np
import pytest
import torch

import paged_ref as P
import test_paged_gpu as T
from adaptive_head_kv_gb300 import fastgen as fg
from test_paged_gpu import CODE, DT, PUNCT, SPECIAL, Setup, dev, f64, gen, table

pytestmark = pytest.mark.gpu


class Step(Setup):
    """Caches that also keep their rows' weights (scores)."""

    prefix = None

    def with_scores(self, seed):
        n = self.cache.c.n_pages
        x = torch.rand(n, 64, generator=gen(seed)) * 3
        x[x < 0.3] = 0.0
        x[x > 2.9] = float("inf")
        self.scores = dev(x)
        return self

    scores = None

    def decode(self, q, ids, k, v, pos, rope=None, out=None, reuse=None):
        ws = reuse
        if ws is None:
            need = fg.fastgen_decode_q8_ex_workspace_bytes(
                self.p, self.cache, self.prefix and self.prefix.cache, self.scores is not None)
            ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        if out is None:
            out = torch.full((self.G, self.d), 3.5, dtype=DT[self.dtype], device="cuda")
        new = [None if x is None else dev(x) for x in (k, v, ids)]
        fg.fastgen_decode_attn_q8_ex(
            self.p, self.cache, self.prefix and self.prefix.cache, self.scores, dev(q), new[0],
            new[1], new[2], self.special, self.punct, dev(pos, torch.int32), rope, out, ws, self.err)
        return out

    def kv(self, c, t):
        """K, V, V's exponents of all rows that cache c's queries see, segment rows of its own
        first, and how many rows are a prompt's."""
        k, v, e = self.ref[c].kv(t)
        if self.prefix is None:
            return k, v, e, 0
        pk, pv, pe = self.prefix.ref[c % self.hl].kv(t)
        return (np.concatenate([k, pk]), np.concatenate([v, pv]), np.concatenate([e, pe]), len(pk))

    def check_out(self, out, q, pos, turn=None, idle=3.5, scores=None):
        """scores [n_pages, 64]: those before the step, whose weights are checked as well."""
        got, hkv = f64(out), self.p.Hkv or self.p.H
        gpu = P.GpuPages(self.cache) if scores is not None else None
        want_s = f64(scores).reshape(-1) if scores is not None else None
        off_s = np.zeros_like(want_s) if scores is not None else None
        for c in range(self.gk):
            b, rows = c // self.hl, self.ref[c].rows
            g0 = (c // hkv) * self.p.H + (c % hkv) * self.R
            if pos[b] < 0:
                assert (got[g0: g0 + self.R] == idle).all()
                continue
            at = np.arange(0)
            if scores is not None and rows:
                pages = gpu.pages(c, False)[: -(-rows // 64)]
                at = (pages[:, None] * 64 + np.arange(64)).reshape(-1)[:rows]
                fresh = gpu.pos[pages].reshape(-1)[:rows] == pos[b]
                if self.new is not None and fresh[-1]:  # the row that the step appended
                    want_s[at[-1]] = np.inf if int(self.new[b]) in SPECIAL else 0.0
            k, v, ev, shared = self.kv(c, pos[b])
            for g in range(g0, g0 + self.R):
                qq = f64(q[g])
                if turn:
                    qq = turn(qq, pos[b])
                want, weight, products, floor = P.attend(qq, k, v, ev, 1 / np.sqrt(self.d))
                # a prompt's weights enter as f16 of 2^7 w_j / max w: steps of 2^-24 below, so
                # 2^-32 of the largest, 2^8 of the other path's; each of a few corrections of the
                # maximum on the way and each part joined adds 2^-23 to what it scales
                bound = P.decode_bound(want, weight, products, floor * (256 if shared else 1),
                                       self.dtype) + (2.0 ** -19 * weight if shared else 0)
                assert (np.abs(got[g] - want) <= bound).all(), (
                    g, np.abs(got[g] - want).max(), bound.min(), len(k), shared)
                if len(at):
                    s = (k @ qq) / np.sqrt(self.d)
                    p = np.exp(s - s.max())
                    p = (p / p.sum())[:rows]
                    # as in decode_bound: the score moves a weight and the sum; exponentials 2^-19
                    ds = products * ((2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -21) + 2.0 ** -20)
                    want_s[at] += p
                    off_s[at] += p * (np.expm1(2 * ds) + 2.0 ** -18)
        if scores is not None:
            now = f64(self.scores).reshape(-1)
            off = np.isfinite(want_s)
            assert np.array_equal(now[~off], want_s[~off])
            # R <= 8 sums and the addition in 32 bits, each 2^-24 of at most the result; below 2^-126
            # nothing is promised
            off_s = off_s[off] + 9 * 2.0 ** -24 * np.abs(want_s[off]) + 2.0 ** -126
            err = np.abs(now[off] - want_s[off])
            assert (err <= off_s).all(), (err.max(), (err / off_s).max())

    new = None

    def step(self, seed, pos, scale=1.0, rope=None, turn=None, token=True, check=True, **kw):
        """A step and its check."""
        q = (torch.randn(self.G, self.d, generator=gen(seed)) * scale).to(DT[self.dtype])
        ids, k, v = self.tokens(seed, 1) if token else (None, None, None)
        self.new = ids[:, 0] if token else None
        before = None if self.scores is None else self.scores.clone()
        out = self.decode(q, ids, k, v, pos, rope, **kw)
        if token:
            self.ref_append(ids, k, v, pos, turn=turn)
        if check:
            self.check(rotated=turn is not None, empty=False)
        self.check_out(out, q, pos, turn, scores=before)
        return out


class Fork(Step):
    """B sequences behind a prompt (a Setup of one sequence)."""

    def __init__(self, prefix, B, max_new=40, pages=None):
        a = prefix.p
        self.prefix, self.max_new = prefix, max_new
        self.p = fg.Params(B, a.L, a.H, a.n, a.d, a.dtype, 0.95, a.r_l, 0.3, 0.0, a.Hkv)
        self.B, self.n, self.d, self.dtype = B, prefix.n, prefix.d, prefix.dtype
        self.G, self.gk, self.R, self.hl, self.w = (
            B * prefix.G, B * prefix.gk, prefix.R, prefix.hl, prefix.w)
        self.special, self.punct = prefix.special, prefix.punct
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        self.cache = fg.PagedCache(
            self.p, None, None, None, None,
            torch.full((fg.fastgen_paged_fork_table_len(self.p, max_new),), -7, **i32),
            torch.zeros(self.gk, 6, **i32), torch.full((self.gk,), 9, **i32), torch.zeros(1, **i32))
        self.info = fg.fastgen_paged_fork(self.p, prefix.cache, max_new, self.cache)
        self.fill = 0x35
        self.set_pages(max(1, self.info.max_pages if pages is None else self.info.pages + pages))
        self.ref = [self.empty(c) for c in range(self.gk)]
        fg.fastgen_paged_clear(self.p, self.cache, self.err)

    def empty(self, c):
        r = P.RefCache(self.prefix.ref[c % self.hl].policy, self.w,
                       (self.max_new + 63) // 64 * 64 or 64, self.d)
        for side in (*r.seg.values(), *r.ring.values()):
            side.codes[:] = 0.8125
        return r

    def tokens(self, seed, m):
        return Setup.tokens(self, seed, m)


def fork(seed, B, max_new=40, pages=None, **kw):
    s = Setup(seed, B=1, max_new=1, **kw)
    s.compact()
    return Fork(s, B, max_new, pages)


# --------------------------------------------------------------- the prompt
@pytest.mark.parametrize("kw", T.SHAPES[:3])
def test_fork_lays_out_empty_caches(kw):
    if "B" in kw:
        kw = {k: x for k, x in kw.items() if k != "B"}
    f = fork(1, 3, 130, **kw)
    gpu = f.check(empty=False)
    used, most = [], 0
    for c, r in enumerate(f.ref):
        seg, ring = gpu.pages(c, False), gpu.pages(c, True)
        assert len(seg) == 3 and (seg == -1).all() and len(ring) == -(-r.w // 64)
        used += list(ring)
        most += 3 + len(ring)
        e = gpu.e[ring].reshape(-1, 2)
        assert (e == P.E_MIN).all() and (gpu.pos[ring] == -1).all()
    assert used == list(range(len(used)))
    assert (f.info.pages, f.info.max_pages, f.info.table_used) == (len(used), most, most)
    assert (f.cache.rows == 0).all() and (f.cache.rows_out == 0).all()
    # a step's rows, then cleared: the pages stay
    for t in range(f.n, f.n + 70):
        ids, k, v = f.tokens(t, 1)
        f.append(ids, k, v, [t, t + 1, -1])
    taken = int(f.cache.next_page.item())
    before = f.cache.page_table.clone()
    assert taken > len(used)
    fg.fastgen_paged_clear(f.p, f.cache, f.err)
    assert torch.equal(before, f.cache.page_table) and int(f.cache.next_page.item()) == taken
    for c in range(f.gk):
        f.ref[c] = f.empty(c)
        f.ref[c].seg["k"].codes[:] = 0
    gpu = f.check(empty=False)
    for st in range(3):
        f.step(st, [f.n, f.n + 5, f.n + 2] if st == 0 else [f.n + st, -1, -1])
    assert int(f.err.item()) == 0


SHARED = [
    (3, dict()),
    (1, dict(n=1, L=1)),
    (2, dict(n=2, d=64, L=1, dtype="fp32")),
    (5, dict(H=8, Hkv=2, n=333)),
    (7, dict(H=8, Hkv=4, n=65, d=64)),
    (3, dict(H=8, Hkv=1, L=3, n=200, dtype="fp32")),
    (17, dict(H=8, Hkv=1, L=1, n=700)),              # 136 queries a cache: two tiles
    (33, dict(H=8, Hkv=1, L=1, n=450, d=64)),        # 264: three tiles, the last alone
    (33, dict(H=8, Hkv=1, L=1, n=300, dtype="fp32")),
    (130, dict(H=2, L=1, n=260)),                    # groups of 1, two tiles
    (129, dict(H=1, L=1, n=1000, dtype="fp32", d=64)),
    (4, dict(n=64, r_l=0.01)),
    (3, dict(n=129, r_l=0.0)),
    (3, dict(n=40, r_l=1.0, d=64)),
    (6, dict(n=1300, L=1, r_l=0.45)),
    (9, dict(n=2600, L=1, H=4, Hkv=1, policies=[4])),
    (2, dict(n=150, L=14, H=8, Hkv=8, policies=[4, 3, 0, 2])),
    (16, dict(n=90, L=8, H=8)),                      # small own caches, many
    (11, dict(n=33, L=16, H=16, Hkv=8, d=64, dtype="fp32")),
]


@pytest.mark.parametrize("B,kw", SHARED)
def test_shared_steps(B, kw):
    f = fork(2, B, 12, **kw)
    if B in (3, 5, 17):
        f.with_scores(1)
    before = [x.clone() for x in (f.prefix.cache.k_pages, f.prefix.cache.v_pages,
                                  f.prefix.cache.exps, f.prefix.cache.pos, f.prefix.cache.rows)]
    for st in range(5):
        pos = np.array([f.n + st + 3 * (b % 4) for b in range(B)])
        if st in (1, 3) and B > 1:  # idle ones first, last, several
            pos[[0, -1] if st == 1 else slice(1, None, 2)] = -1
        f.step(100 + st, pos.tolist(), scale=(1, 3, 0.01)[st % 3], check=st in (0, 4))
    f.step(9, [f.n + 12 + 3 * (b % 4) for b in range(B)], token=False)
    for x, y in zip(before, (f.prefix.cache.k_pages, f.prefix.cache.v_pages, f.prefix.cache.exps,
                             f.prefix.cache.pos, f.prefix.cache.rows)):
        assert torch.equal(x, y)
    assert int(f.err.item()) == 0


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d,rot,dtype", [(128, 128, "bf16"), (64, 64, "fp32"), (128, 48, "fp32"),
                                         (64, 16, "bf16")])
def test_shared_steps_rotate(half, d, rot, dtype):
    inv, turns = table(rot)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    turn = lambda x, at: P.rotate(x, at, inv, half)
    f = fork(7, 3, H=4, Hkv=2, d=d, dtype=dtype, n=70).with_scores(2)
    for st in range(3):
        f.step(st, [70 + st, 75 + st, 100000 + st], rope=rope, turn=turn)
    assert int(f.err.item()) == 0


def test_windows_that_slide_off_the_prompt_and_empty_prompts():
    """Ring rows of the prompt leave the window as a sequence goes on; where neither side has a row
    the output is zero."""
    f = fork(12, 4, L=2, H=4, n=100, policies=[0, 4, 3, 0])
    w = f.w
    for pos in ([99, 99 + w - 1, 99 + w, 5000], [-1, -1, 99 + w // 2, -1], [-1] * 4):
        out = f.step(1, pos, token=False)
        if pos[0] == 99:
            none = [c for c in range(f.gk) if len(f.kv(c, pos[c // f.hl])[0]) == 0]
            assert none and (out[none] == 0).all()
    assert int(f.err.item()) == 0


def test_a_prompt_with_no_row_at_all():
    f = fork(13, 3, L=1, H=4, n=50, policies=[0], r_l=0.2)
    for r, c in zip(f.prefix.ref, range(f.hl)):
        r.rows = 0
    f.prefix.cache.rows.zero_()
    out = f.step(1, [50, 51, 52], token=False)
    assert (out == 0).all()
    f.step(2, [50, 51, -1])
    f.step(3, [51, -1, 52])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [3, 150])
def test_nan_outside_the_prompt_and_inside_it(dtype, B):
    """Rows that are not in the prompt's caches may hold NaN; a NaN inside stays with its heads, in a
    ring also with the queries whose window has the row."""
    s = Setup(13, L=1, H=5, n=100, dtype=dtype, max_new=1)
    s.fill = 0x7F
    s.set_pages(s.info.max_pages)
    s.compact()
    f = Fork(s, B)
    pos = [100 + b % 7 for b in range(B)]
    q = torch.randn(f.G, f.d, generator=gen(1)).to(DT[dtype])
    f.check_out(f.decode(q, None, None, None, pos), q, pos)
    gpu = P.GpuPages(s.cache)
    page, ring = int(gpu.pages(4, False)[0]), int(gpu.pages(3, True)[0])
    s.cache.k_pages[page, 3, 5] = 0x7F
    # the oldest ring row: in the windows of some of the sequences
    old = int(np.min(s.ref[3].ring_pos[s.ref[3].ring_pos >= 0]))
    s.cache.v_pages[ring, old % s.w, 7] = 0x7F
    assert old % s.w < 64
    pos = [old + s.w - 2 + b % 4 for b in range(B)]  # seen while pos < old + w
    out = f.decode(q, None, None, None, pos).view(B, 5, f.d)
    assert torch.isnan(out[:, 4]).all() and torch.isfinite(out[:, :3]).all()
    sees = torch.tensor([p < old + s.w for p in pos], device="cuda")
    assert sees.any() and not sees.all()
    assert torch.isnan(out[sees, 3]).all() and torch.isfinite(out[~sees, 3]).all()
    # in a segment's V: that column of that head
    s.cache.k_pages[page, 3, 5] = 0
    s.cache.v_pages[page, 3, 5] = 0x7F
    out = f.decode(q, None, None, None, pos).view(B, 5, f.d)
    assert torch.isnan(out[:, 4, 5]).all()
    keep = torch.arange(f.d, device="cuda") != 5
    assert torch.isfinite(out[:, 4][:, keep]).all() and torch.isfinite(out[:, :3]).all()


def test_large_exponents_of_the_prompt():
    def plant(s):
        s.V[:, ::31] *= 2.0 ** 60
        s.V[:, 1::31] *= 2.0 ** -60
        s.K[:, 2::37] *= 2.0 ** -40
        s.K[:, 50] *= 30.0
    for dtype in ("bf16", "fp32"):
        for B in (3, 70):
            f = fork(14, B, L=1, H=8, Hkv=4, n=210, dtype=dtype, policies=[4, 4, 3, 3, 2],
                     plant=plant)
            q = torch.randn(f.G, f.d, generator=gen(1)).to(DT[dtype])
            for scale in (1.0, 2.0 ** -30, 2.0 ** 5):
                qs = (q.float() * scale).to(DT[dtype])
                pos = [210 + b % 3 for b in range(B)]
                f.check_out(f.decode(qs, None, None, None, pos), qs, pos)


def test_scores_that_climb_along_the_prompt():
    """Rows in order of their score, so that the running maximum moves at every page."""
    for dtype in ("bf16", "fp32"):
        for down in (False, True):
            def plant(s):
                s.K[:] = 0.02 * s.K.float().to(s.K.dtype)
                ramp = torch.linspace(0, 8, s.n)
                s.K[..., 0] = (ramp.flip(0) if down else ramp).to(s.K.dtype)
            f = fork(15, 3, L=1, H=2, n=1000, dtype=dtype, policies=[4], plant=plant)
            q = torch.randn(f.G, f.d, generator=gen(1)).to(DT[dtype])
            q[:, 0] = 100.0  # up to 70 of score
            pos = [1000] * 3
            f.check_out(f.decode(q, None, None, None, pos), q, pos)


def test_bad_pages_of_the_prompt_are_flagged_not_followed():
    f = fork(16, 3, L=1, H=5, n=200).with_scores(1)
    pre = f.prefix.cache
    keep = [x.clone() for x in (pre.page_table, pre.caches, pre.rows)]
    q = torch.randn(f.G, f.d, generator=gen(1)).to(DT[f.dtype])

    def flagged():
        out = f.decode(q, None, None, None, [200, 201, 202])
        assert fg.fastgen_read_error(f.err) == fg.FG_EINVAL
        assert torch.isfinite(out).all()
        for x, y in zip((pre.page_table, pre.caches, pre.rows), keep):
            x.copy_(y)
        f.err.zero_()

    first = int(pre.caches[4, 2])
    for bad in (pre.c.n_pages, 1 << 30, -5):
        pre.page_table[first + 1] = bad
        flagged()
    for col, bad in ((2, -1), (2, 1 << 30), (4, 1 << 30), (3, 0), (1, 1 << 20), (1, -3)):
        pre.caches[3:, col] = bad
        flagged()
    for bad in (1 << 30, -9):
        pre.rows[4] = bad
        flagged()


# ------------------------------------------------------------- the weights
@pytest.mark.parametrize("kw", T.SHAPES + [dict(H=4, Hkv=2, n=700, L=1),
                                           dict(n=2600, L=1, H=4, Hkv=1, policies=[4, 3]),
                                           dict(H=8, Hkv=1, n=300, L=2, B=2),
                                           dict(B=2, L=16, H=32, n=70),
                                           dict(B=4, L=16, H=32, Hkv=16, n=20, dtype="fp32")])
def test_steps_that_keep_weights(kw):
    s = Step(11, max_new=8, **kw)
    s.compact()
    s.with_scores(3)
    for st in range(4):
        pos = [s.n + st + 2 * b if st % 3 != 1 or b == 0 else -1 for b in range(s.B)]
        s.step(200 + st, pos, scale=1 + st, check=st == 3)
    s.step(5, [s.n + 20] * s.B, token=False)
    assert int(s.err.item()) == 0


def test_weights_of_other_rows_stay():
    """Pages that no active segment uses, rows behind the last, rings, idle sequences."""
    s = Step(18, B=3, L=1, H=4, n=90)
    s.compact()
    s.with_scores(1)
    s.scores[:] = torch.rand(s.scores.shape, generator=gen(4)).cuda()
    before = s.scores.clone()
    s.step(3, [90, -1, 91])
    gpu, touched = P.GpuPages(s.cache), torch.zeros_like(s.scores, dtype=torch.bool)
    for c, r in enumerate(s.ref):
        if c // s.hl != 1:
            for i in range(r.rows):
                touched[int(gpu.pages(c, False)[i // 64]), i % 64] = True
    assert torch.equal(s.scores[~touched], before[~touched]) and touched.any()


def test_without_options_the_step_is_the_plain_one():
    a, b = (cls(19, B=2, L=2, H=8, Hkv=4, n=300) for cls in (Setup, Step))
    for s in (a, b):
        s.compact()
    for st in range(3):
        ids, k, v = a.tokens(st, 1)
        q = torch.randn(a.G, a.d, generator=gen(st)).to(torch.bfloat16)
        pos = [300 + st, -1 if st == 1 else 310 + st]
        x, y = (s.decode(q, ids, k, v, pos) for s in (a, b))
        a.ref_append(ids, k, v, pos)
        b.ref_append(ids, k, v, pos)
        a.check_out(x, q, pos)
        b.check_out(y, q, pos)
    b.check()


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2)])
def test_scores_that_rows_start_with(H, Hkv):
    s = Step(20, B=2, L=2, H=H, Hkv=Hkv, n=130, max_new=100)
    s.compact()
    g = gen(5)
    s.scores = torch.full((s.cache.c.n_pages, 64), 7.5, device="cuda")
    ids = torch.randint(100, 300, (2, 130), generator=g, dtype=torch.int32)
    ids[:, 0], ids[1, 129] = SPECIAL[0], SPECIAL[1]
    col = torch.rand(s.G, 130, generator=g)
    args = lambda *x: fg.fastgen_scores_q8(s.p, s.cache, s.scores, *x, s.special, s.err)
    args(dev(col), dev(ids), None, None)

    def expect(want, colsum, ids, pos, n_new):
        gpu = P.GpuPages(s.cache)
        for c, r in enumerate(s.ref):
            b = c // s.hl
            g0 = (c // Hkv) * H + (c % Hkv) * s.R
            for i in range(r.rows):
                j = int(r.seg_pos[i]) - pos[b]
                if pos[b] < 0 or not 0 <= j < n_new[b]:
                    continue
                at = (int(gpu.pages(c, False)[i // 64]), i % 64)
                y = np.float32(0)
                for x in range(s.R if colsum is not None else 0):
                    y += colsum[g0 + x, j].numpy()  # in the heads' order, 32 bits
                want[at] = np.inf if int(ids[b, j]) in SPECIAL else y
        return want

    want = expect(np.full((s.cache.c.n_pages, 64), 7.5, dtype=np.float32), col, ids, [0, 0], [130] * 2)
    assert np.array_equal(s.scores.cpu().numpy(), want)
    new, k, v = s.tokens(6, 40)
    for pos, n_new in (([130, 200], [40, 0]), ([-1, 200], [40, 33])):
        s.append(new, k, v, pos, n_new)
        s.ref_append(new, k, v, pos, n_new)
        args(None, dev(new), dev(n_new, torch.int32), dev(pos, torch.int32))
        want = expect(want, None, new, pos, n_new)
        assert np.array_equal(s.scores.cpu().numpy(), want)
    assert int(s.err.item()) == 0


# ------------------------------------------------------------------ the cut
def cut(ref, score, budget, recent, t):
    """The reference's cut of one cache; score [rows], changed in place.  Returns the moves."""
    rows = ref.rows
    if t < 0 or rows <= budget:
        return []
    s = np.where(score > 0, score, 0.0)  # NaN and negative ones too
    new = (ref.seg_pos[:rows] <= t) & (ref.seg_pos[:rows] > t - recent)
    order = sorted(range(rows), key=lambda r: (not new[r], -s[r], r))
    stay = set(order[:budget])
    holes = [r for r in range(budget) if r not in stay]
    moves = list(zip(holes, sorted(r for r in stay if r >= budget)))
    for x in "kv":
        side = ref.seg[x]
        vals = {dst: side.values([src])[0] for dst, src in moves}
        if moves:
            side.put([d for d, _ in moves], [vals[d] for d, _ in moves], lambda b: False)
    for d, src in moves:
        ref.seg_pos[d], score[d] = ref.seg_pos[src], score[src]
    ref.rows = budget
    return moves


def check_cut(s, budget, recent, pos, aliased=True):
    """Cuts on the GPU and in the reference, compares everything.  s.scores are there."""
    gpu = P.GpuPages(s.cache)
    sc = s.scores.cpu().numpy().copy()
    want = sc.copy()
    total = 0
    for c, r in enumerate(s.ref):
        rows = r.rows
        pages = gpu.pages(c, False)[: -(-rows // 64)]
        at = (pages[:, None] * 64 + np.arange(64)).reshape(-1)[:rows]
        mine = want.reshape(-1)[at]
        total += len(cut(r, mine, budget, recent, pos[c // s.hl]))
        want.reshape(-1)[at] = mine
    ws = torch.full((fg.fastgen_evict_q8_workspace_bytes(s.p, budget),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    fg.fastgen_evict_q8(s.p, s.cache, s.scores, budget, recent, dev(pos, torch.int32), ws, s.err)
    assert np.array_equal(s.scores.cpu().numpy(), want, equal_nan=True)
    return total


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,budget,recent", [(1, 16, 0), (16, 16, 16), (17, 16, 0), (150, 16, 16),
                                             (150, 64, 10), (150, 144, 0), (333, 208, 37),
                                             (1500, 1024, 100), (1500, 1024, 1024)])
def test_cut(n, budget, recent, d):
    s = Step(31, B=2, L=1, H=5, n=n, d=d, dtype="fp32" if d == 64 else "bf16",
             policies=[4, 4, 3, 2, 1]).with_scores(7)
    s.compact()
    for pos in ([n - 1, -1], [n - 1, n - 1], [n + 3, n - 1]):
        check_cut(s, budget, recent, pos)
        s.check()
    assert int(s.err.item()) == 0


def test_cut_ties_and_odd_scores():
    """Equal scores, zeros, negative, NaN, infinities, subnormals."""
    for values in ([1.0], [0.0, -1.0, float("nan"), -float("inf")], [float("inf")],
                   [2.0 ** -149, 0.0, 2.0 ** -140], [1.0, 1.0 + 2.0 ** -23, 1.0 + 2.0 ** -22],
                   [float("inf"), float("nan"), 3e38, -0.0, 1.0]):
        s = Step(32, L=1, H=3, n=400, policies=[4, 4, 3])
        s.compact()
        x = torch.randint(0, len(values), (s.cache.c.n_pages, 64), generator=gen(1))
        s.scores = dev(torch.tensor(values)[x])
        assert check_cut(s, 208, 21, [399]) > 0
        s.check()


def test_cut_of_a_few_long_caches():
    """More rows than the small form holds, and than shared memory holds."""
    for n, budget, recent in ((9000, 4096, 200), (50000, 16000, 5000)):
        s = Step(33, L=1, H=2, n=n, d=64, policies=[4, 3], max_new=4).with_scores(2)
        s.compact()
        s.scores *= 0.001
        assert check_cut(s, budget, recent, [n - 1]) > 0
        s.check()
        assert int(s.err.item()) == 0


def test_cut_of_blocks_of_many_sizes():
    """Rows that come to blocks of smaller exponents, and of larger ones."""
    def plant(s):
        size = 2.0 ** torch.randint(-30, 30, (s.n,), generator=gen(9)).double()
        s.K[:] = (s.K.double() * size[:, None]).to(s.K.dtype)
        s.V[:] = (s.V.double() * size.flip(0)[:, None]).to(s.V.dtype)
        s.V[:, 77, 3], s.K[:, 380, 5], s.V[:, 381, 6] = float("nan"), float("inf"), float("nan")
    s = Step(34, L=2, H=4, n=400, policies=[4, 4, 3, 2], plant=plant, dtype="fp32").with_scores(3)
    s.compact()
    check_cut(s, 96, 30, [399])
    s.check()
    check_cut(s, 48, 7, [399])
    s.check()


def test_cut_reads_rows_and_writes_rows_out():
    s = Step(35, L=1, H=4, n=200, policies=[4, 3, 0, 2]).with_scores(3)
    s.compact()
    before = s.cache.rows.clone()
    s.cache.rows_out = torch.full_like(before, 55)
    s.cache.c.rows_out = s.cache.rows_out.data_ptr()
    check_cut(s, 64, 10, [199])
    assert torch.equal(s.cache.rows, before)
    assert s.cache.rows_out.tolist() == [min(int(x), 64) for x in before]
    s.check()


def test_cut_bad_pages_are_flagged_not_followed():
    s = Step(36, L=1, H=5, n=300, policies=[4]).with_scores(3)
    s.compact()
    ws = torch.empty(fg.fastgen_evict_q8_workspace_bytes(s.p, 64), dtype=torch.uint8, device="cuda")
    keep = [x.clone() for x in (s.cache.page_table, s.cache.caches, s.cache.rows)]
    first = int(s.cache.caches[2, 2])
    plants = [(s.cache.page_table, first + i, bad) for i in (0, 1, 4) for bad in (1 << 30, -5)]
    plants += [(s.cache.caches[2:3, j], 0, bad) for j, bad in ((2, -1), (2, 1 << 30), (3, 0))]
    plants += [(s.cache.caches[2:3, 1], 0, bad) for bad in (1 << 20, -1)]  # ring slots
    plants += [(s.cache.rows, 2, bad) for bad in (1 << 30, -9)]
    for x, i, bad in plants:
        x[i] = bad
        fg.fastgen_evict_q8(s.p, s.cache, s.scores, 64, 5, dev([299], torch.int32), ws, s.err)
        assert fg.fastgen_read_error(s.err) == fg.FG_EINVAL
        s.err.zero_()
        fg.fastgen_scores_q8(s.p, s.cache, s.scores, None, dev(torch.zeros(1, 300), torch.int32),
                             None, None, s.special, s.err)
        for y, z in zip((s.cache.page_table, s.cache.caches, s.cache.rows), keep):
            y.copy_(z)
        s.err.zero_()


# -------------------------------------------------------------- calls less usual
def test_steps_repeat_bit_for_bit():
    outs = []
    for _ in range(3):
        f = fork(17, 40, L=2, H=8, Hkv=2, n=900, policies=[4, 3]).with_scores(1)
        for st in range(2):
            out = f.step(st, [900 + st] * 40, check=False) if not outs else None
            if out is None:
                q = torch.randn(f.G, f.d, generator=gen(st)).to(torch.bfloat16)
                ids, k, v = f.tokens(st, 1)
                out = f.decode(q, ids, k, v, [900 + st] * 40)
        gpu, sc = P.GpuPages(f.cache), f.scores.cpu()  # by rows: pages are taken in any order
        outs.append((out.clone(), torch.cat([sc[gpu.pages(c, False)[:1]][0, : gpu.rows[c]]
                                             for c in range(f.gk)])))
    assert len(outs[0][1]) > 100
    for x, y in zip(outs[0] * 2, outs[1] + outs[2]):
        assert torch.equal(x, y)


def test_two_forks_of_one_prompt_on_two_streams():
    """Two batches read one prompt at the same time, each with its own workspace."""
    pre = Setup(40, B=1, L=2, H=8, Hkv=2, n=1200, max_new=1, policies=[4, 3, 4, 2])
    pre.compact()
    a, b = Fork(pre, 20), Fork(pre, 3)
    torch.cuda.synchronize()
    streams, held = [torch.cuda.Stream() for _ in range(2)], []
    for st in range(4):
        for f, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                q = torch.randn(f.G, f.d, generator=gen(st)).to(torch.bfloat16)
                ids, k, v = f.tokens(st, 1)
                pos = [1200 + st] * f.B
                held.append((f, f.decode(q, ids, k, v, pos), q, ids, k, v, pos))
    torch.cuda.synchronize()
    for f, out, q, ids, k, v, pos in held:
        f.ref_append(ids, k, v, pos)
        f.check_out(out, q, pos)
    a.check(empty=False)
    b.check(empty=False)


def test_captured_steps_share_a_workspace():
    """A step behind a prompt, one with weights and a cut, captured with one workspace, replayed in
    turn while rows come and the positions move on the device."""
    f = fork(41, 5, 100, L=1, H=4, Hkv=2, n=300, policies=[4, 3]).with_scores(1)
    s = Step(42, L=1, H=4, n=60, policies=[4, 3, 4, 1], max_new=100).with_scores(2)
    s.compact()
    need = max(fg.fastgen_decode_q8_ex_workspace_bytes(f.p, f.cache, f.prefix.cache, 1),
               fg.fastgen_decode_q8_ex_workspace_bytes(s.p, s.cache, None, 1),
               fg.fastgen_evict_q8_workspace_bytes(s.p, 80))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in (f, s):
        ids, k, v = x.tokens(1, 1)
        x.new = ids[:, 0]
        q = torch.randn(x.G, x.d, generator=gen(1)).to(torch.bfloat16)
        io = [dev(y) for y in (q, k, v, ids)] + [dev([x.n] * x.B, torch.int32),
                                                 torch.zeros(x.G, x.d, dtype=torch.bfloat16,
                                                             device="cuda")]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fg.fastgen_decode_attn_q8_ex(x.p, x.cache, x.prefix and x.prefix.cache, x.scores, io[0],
                                         io[1], io[2], io[3], x.special, x.punct, io[4], None, io[5],
                                         ws, x.err)
            if x is s:
                fg.fastgen_evict_q8(x.p, x.cache, x.scores, 80, 5, io[4], ws, x.err)
            io[4] += 1
        graphs.append((x, g, io, (ids, k, v, q)))
    for st in range(70):
        for x, g, io, (ids, k, v, q) in graphs:
            before = x.scores.clone()
            g.replay()
            t = x.n + st
            x.ref_append(ids, k, v, [t] * x.B)
            if x is s:
                # the step's own scores are not seen between the two; the cut only after row 80
                if any(r.rows > 80 for r in s.ref):
                    sc = x.scores.cpu().numpy()
                    assert [int(y) for y in x.cache.rows] == [min(r.rows, 80) for r in s.ref]
                    x.check_out(io[5], q, [t] * x.B)
                    return_rows = P.GpuPages(x.cache)
                    for c, r in enumerate(s.ref):  # go on from what is stored
                        r.rows = int(return_rows.rows[c])
                        if r.rows:
                            got = return_rows.segment(c, False, r.rows)
                            for y in "kv":
                                r.seg[y].codes[:r.rows] = got[y]
                                r.seg[y].e[: -(-r.rows // 16)] = got["e" + y]
                            r.seg_pos[:r.rows] = got["pos"]
                            assert t in got["pos"] or r.policy != P.FULL
                    assert np.isfinite(sc).any()
                    continue
                x.check_out(io[5], q, [t] * x.B, scores=before)
            elif st % 20 == 0 or st == 69:
                x.check_out(io[5], q, [t] * x.B, scores=before)
    f.check(empty=False)
    s.check()
    assert int(f.err.item()) == 0 and int(s.err.item()) == 0


def test_the_largest_groups_and_many_tiles():
    """R B = 1040 queries a cache: nine tiles, the last of 16."""
    f = fork(43, 130, 4, H=8, Hkv=1, L=1, n=500, policies=[4]).with_scores(1)
    f.step(1, [500 + b % 3 for b in range(130)])
    f.step(2, [-1 if b % 3 else 510 for b in range(130)], token=False)


def test_the_step_leaves_its_guards_alone():
    """Outputs, scores and workspace between guard bytes."""
    f = fork(44, 3, L=1, H=8, Hkv=2, n=333, dtype="fp32")
    need = fg.fastgen_decode_q8_ex_workspace_bytes(f.p, f.cache, f.prefix.cache, 1)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((f.G + 2, f.d), 3.5, device="cuda")
    sc = torch.full((f.cache.c.n_pages + 2, 64), 0.25, device="cuda")
    f.scores = sc[1:-1]
    q = torch.randn(f.G, f.d, generator=gen(1))
    f.check_out(f.decode(q, None, None, None, [333] * 3, out=out[1:-1], reuse=ws[256:256 + need]), q,
                [333] * 3)
    assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all()
    assert (out[[0, -1]] == 3.5).all() and (sc[[0, -1]] == 0.25).all()


def lift(s, by):
    """The same caches in the last pages of a pool that is `by` pages larger."""
    c, n = s.cache, s.cache.c.n_pages
    old = [x.clone() for x in (c.k_pages, c.v_pages, c.exps, c.pos)]
    s.set_pages(n + by)
    for x, y in zip((c.k_pages, c.v_pages, c.exps, c.pos), old):
        x[by:] = y
    t = c.page_table
    t.copy_(torch.where(t >= 0, t + by, t))
    c.next_page += by


def same_rows(x, y):
    """Pages, positions and scores of two pools by their tables."""
    tx, ty = x.cache.page_table.long(), y.cache.page_table.long()
    tx, ty = tx[tx >= 0], ty[ty >= 0]
    assert torch.equal(x.cache.rows, y.cache.rows) and len(tx) == len(ty)
    for name in ("k_pages", "v_pages", "exps", "pos"):
        assert torch.equal(getattr(x.cache, name)[tx], getattr(y.cache, name)[ty]), name
    assert torch.equal(x.scores[tx], y.scores[ty])


def test_pages_past_four_gigabytes():
    """Codes and scores that lie past 2^32 bytes of their buffers give what they give before."""
    by = 540000  # pages of 64 x 128 codes: 4.4e9 bytes; a step's scores of groups of 8: 1.1e9
    pair = [fork(45, 9, L=1, H=16, Hkv=2, n=200, policies=[4, 3]) for _ in range(2)]
    lift(pair[1], by)
    lift(pair[1].prefix, by)
    for f in pair:
        f.scores = torch.zeros(f.cache.c.n_pages, 64, device="cuda")
    for st in range(3):
        ids, k, v = pair[0].tokens(st, 1)
        q = torch.randn(pair[0].G, 128, generator=gen(st)).to(torch.bfloat16)
        outs = [f.decode(q, ids, k, v, [200 + st] * 9) for f in pair]
        assert torch.equal(*outs) and float(outs[0].abs().max()) > 0
    same_rows(*pair)
    assert int(pair[1].cache.next_page.item()) > by and int(pair[1].err.item()) == 0
    del f, pair
    pair = [Step(46, L=1, H=8, Hkv=1, n=150, policies=[4]) for _ in range(2)]
    for s in pair:
        s.compact()
    lift(pair[1], by)
    ws = torch.empty(fg.fastgen_evict_q8_workspace_bytes(s.p, 64), dtype=torch.uint8, device="cuda")
    ids, k, v = s.tokens(1, 1)
    q = torch.randn(s.G, 128, generator=gen(1)).to(torch.bfloat16)
    outs = []
    for s in pair:
        s.scores = torch.zeros(s.cache.c.n_pages, 64, device="cuda")
        outs.append(s.decode(q, ids, k, v, [150]))
        fg.fastgen_evict_q8(s.p, s.cache, s.scores, 64, 8, dev([150], torch.int32), ws, s.err)
        assert int(s.err.item()) == 0 and s.cache.rows.tolist() == [64]
    assert torch.equal(*outs)
    same_rows(*pair)


# ------------------------------------------------------------ the whole path
@pytest.mark.parametrize("dtype,H,Hkv,d", [("bf16", 8, 2, 128), ("fp32", 4, 4, 64)])
@pytest.mark.parametrize("own_stream", [False, True])
def test_session_forks_a_prompt_and_keeps_a_budget(dtype, H, Hkv, d, own_stream):
    """A prompt, four continuations of it, turns of several tokens, steps with an idle sequence,
    cuts; a captured step; all of it against the reference."""
    from adaptive_head_kv_gb300.session import PagedSession, make_params

    B, L, n, max_new = 4, 3, 210, 120  # caches of every entry of the shortlist
    stream = torch.cuda.Stream() if own_stream else None
    inv, turns = table(d)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF)
    turn = lambda x, at: P.rotate(x, at, inv, True)
    p = make_params(1, L, H, n, d, dtype, 0.9, 0.3, 0.3, Hkv=Hkv)
    G, gk = L * H, L * Hkv
    g = gen(3)
    Q, K, V = (torch.randn(x, n, d, generator=g).to(DT[dtype]) for x in (G, gk, gk))
    ids = torch.randint(100, 300, (1, n), generator=g, dtype=torch.int32)
    ids[:, 0] = SPECIAL[0]
    pre = PagedSession(p, SPECIAL, PUNCT, 8, rope=rope, guard=True, stream=stream)
    with pytest.raises(ValueError):
        pre.fork(2, 10)  # no prompt yet
    saved = torch.arange(G, dtype=torch.int8) // (H // Hkv) % 5
    given = [dev(x) for x in (Q, K, V, ids)]
    torch.cuda.synchronize()
    pre.prefill_with_policy(*given, saved)
    s = pre.fork(B, max_new, budget=32, recent=8, guard=True)
    for bad in (lambda: s.fork(2, 4), lambda: s.compact(given[1], given[2]), lambda: pre.evict(n),
                lambda: s.prefill(*given), lambda: s.prefill_with_policy(*given, saved)):
        with pytest.raises(ValueError):
            bad()
    torch.cuda.synchronize()

    h, hp = Fork.__new__(Fork), Setup.__new__(Setup)
    keep, pol, w = pre.keep.cpu(), pre.policy.cpu(), int(np.ceil(float(np.float32(0.3)) * n))
    Kr, R = f64(pre._rotated[1]), G // gk
    hp.ref = []
    for c in range(gk):
        g0 = (c // Hkv) * H + (c % Hkv) * R
        st = (keep[g0: g0 + R] == 1).any(0)
        win = (keep[g0: g0 + R] == 2).any(0) & ~st
        r = P.RefCache(int(pol[g0: g0 + R].max()), w, 1024, d)
        r.compact(st.nonzero()[:, 0].tolist(), win.nonzero()[:, 0].tolist(), Kr[c], f64(V[c]))
        hp.ref.append(r)
    hp.p, hp.cache, hp.G, hp.gk, hp.R, hp.hl, hp.d, hp.dtype = p, pre.cache, G, gk, R, gk, d, dtype
    hp.w = w
    hp.check(empty=False)
    h.prefix, h.p, h.cache, h.dtype, h.d, h.n, h.B, h.w = hp, s.p, s.cache, dtype, d, n, B, w
    h.G, h.gk, h.R, h.hl, h.max_new, h.err = B * G, B * gk, R, gk, max_new, s.dev_err
    h.ref = [h.empty(c) for c in range(h.gk)]
    h.scores = s.scores.view(-1, 64)
    assert (h.scores == 0).all()
    h.check(empty=False)

    tok, k, v = h.tokens(7, 40)
    pos, n_new = [n] * B, [40, 11, 0, 33]
    given = [dev(x) for x in (k, v, tok)] + [dev(pos, torch.int32), dev(n_new, torch.int32)]
    torch.cuda.synchronize()
    s.append(*given[:4], n_new=given[4])
    torch.cuda.synchronize()
    h.ref_append(tok, k, v, pos, n_new, turn=turn)
    h.check(rotated=True, empty=False)
    # appended rows start at 0, special tokens' at +inf
    gpu, want = P.GpuPages(s.cache), np.zeros(h.scores.shape, dtype=np.float32)
    for c, r in enumerate(h.ref):
        for i in range(r.rows):
            if int(tok[c // h.hl, r.seg_pos[i] - n]) in SPECIAL:
                want[gpu.pages(c, False)[i // 64], i % 64] = np.inf
    assert np.array_equal(h.scores.cpu().numpy(), want) and np.isinf(want).any()
    s.reschedule()

    at, moved = [n + x for x in n_new], 0
    for st in range(14):
        if st in (3, 9):
            pos = [t - 1 if b != 1 else -1 for b, t in enumerate(at)]
            before = h.scores.cpu().numpy().copy()
            gpu, want = P.GpuPages(s.cache), before.copy()
            for c, r in enumerate(h.ref):
                rows = r.rows
                pages = gpu.pages(c, False)[: -(-rows // 64)]
                to = (pages[:, None] * 64 + np.arange(64)).reshape(-1)[:rows]
                mine = want.reshape(-1)[to]
                moved += len(cut(r, mine, 32, 8, pos[c // h.hl]))
                want.reshape(-1)[to] = mine
            posd = dev(pos, torch.int32)
            torch.cuda.synchronize()
            s.evict(posd)
            torch.cuda.synchronize()
            assert np.array_equal(h.scores.cpu().numpy(), want)
            h.check(empty=False)
        pos = [t if (st + b) % 5 else -1 for b, t in enumerate(at)]
        q = torch.randn(h.G, d, generator=gen(60 + st)).to(DT[dtype])
        tok, k, v = h.tokens(80 + st, 1)
        h.new = tok[:, 0]
        before = h.scores.clone()
        out = torch.full((h.G, d), 3.5, dtype=DT[dtype], device="cuda")
        given = [dev(x) for x in (q, k, v, tok)] + [dev(pos, torch.int32)]
        torch.cuda.synchronize()
        if st < 12:
            s.decode(*given, out=out)
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                s.decode(*given, out=out)
            graph.replay()
        torch.cuda.synchronize()
        h.ref_append(tok, k, v, pos, turn=turn)
        h.check(rotated=True, empty=False)
        h.check_out(out, q, pos, turn, scores=before)
        at = [t + (p >= 0) for t, p in zip(at, pos)]
    assert moved > 0
    for x in (pre, s):
        assert fg.fastgen_read_error(x.dev_err) == fg.FG_OK
        assert x.check_guards() == 0


def test_session_scores_start_with_the_column_sums():
    from adaptive_head_kv_gb300.session import PagedSession, make_params

    B, L, H, Hkv, n, d = 2, 1, 4, 2, 100, 64
    p = make_params(B, L, H, n, d, "bf16", 0.9, 0.3, 0.3, Hkv=Hkv)
    g = gen(4)
    Q, K, V = (dev(torch.randn(x, n, d, generator=g).to(torch.bfloat16)) for x in (8, 4, 4))
    ids = torch.randint(100, 300, (B, n), generator=g, dtype=torch.int32)
    ids[:, 0] = SPECIAL[0]
    ids = dev(ids)
    s = PagedSession(p, SPECIAL, PUNCT, 30, budget=32, recent=4, guard=True)
    for way in (lambda: s.prefill(Q, K, V, ids),
                lambda: s.prefill_with_policy(Q, K, V, ids, torch.full((8,), 4, dtype=torch.int8))):
        way()
        gpu, sc = P.GpuPages(s.cache), s.scores.view(-1, 64).cpu().numpy()
        col = s.colsum.cpu().numpy().reshape(4, 2, n)
        full = way.__code__.co_names[0] == "prefill"
        for c in range(4):
            rows = int(gpu.rows[c])
            got = gpu.segment(c, False, rows)["pos"] if rows else []
            for i, j in enumerate(got):
                want = np.inf if int(ids[c // 2, j]) in SPECIAL else (
                    np.float32(col[c, 0, j]) + col[c, 1, j] if full else 0.0)
                assert sc[gpu.pages(c, False)[i // 64], i % 64] == want
    assert (s.cache.rows == n).all()
    before = s.scores.clone()
    s.evict(-1)
    assert (s.cache.rows == n).all() and torch.equal(s.scores, before)
    s.evict(n - 1)
    assert (s.cache.rows == 32).all()
    q = dev(torch.randn(8, d, generator=g).to(torch.bfloat16))
    k, v = (dev(torch.randn(4, d, generator=g).to(torch.bfloat16)) for _ in range(2))
    out = s.decode(q, k, v, ids[:, 5].contiguous(), n)
    assert torch.isfinite(out).all() and (s.cache.rows == 33).all()
    assert fg.fastgen_read_error(s.dev_err) == fg.FG_OK and s.check_guards() == 0


def test_a_captured_cut_of_a_pool_that_was_replaced_does_nothing_and_says_so():
    """A later prompt wants more pages: step and cut captured before leave the new caches, the new
    scores and what the old pool's memory holds now alone; forks of the prompt before see no rows of
    it, and say so."""
    from adaptive_head_kv_gb300.session import PagedSession, make_params

    L, H, n, d = 1, 4, 200, 64
    p = make_params(1, L, H, n, d, "bf16", 0.9, 0.3, 0.3)
    g = gen(6)
    Q, K, V = (dev(torch.randn(4, n, d, generator=g).to(torch.bfloat16)) for _ in range(3))
    ids = dev(torch.randint(100, 300, (1, n), generator=g, dtype=torch.int32))
    s = PagedSession(p, SPECIAL, PUNCT, 60, budget=16, recent=4)
    s.prefill_with_policy(Q, K, V, ids, torch.tensor([3, 0, 0, 3], dtype=torch.int8))
    f = s.fork(2, 8)
    pos = dev([n], torch.int32)
    step = [dev(torch.randn(4, d, generator=g).to(torch.bfloat16)) for _ in range(3)]
    tok = dev([5], torch.int32)
    s.decode(*step, tok, pos)
    s.evict(pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    out = torch.full((4, d), 3.5, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(graph):
        s.decode(*step, tok, pos, out=out)
        s.evict(pos)
    graph.replay()
    assert fg.fastgen_read_error(s.dev_err) == fg.FG_OK
    old = s.cache
    s.prefill_with_policy(Q, K, V, ids, torch.full((4,), 4, dtype=torch.int8))
    assert s.cache is not old and (s.cache.rows == n).all()
    before = [x.clone() for x in (s.cache.k_pages, s.cache.rows, s.cache.page_table, s.scores)]
    graph.replay()
    assert fg.fastgen_read_error(s.dev_err) == fg.FG_EINVAL
    s.dev_err.zero_()
    s.ews.zero_()
    fg.fastgen_evict_q8(s.p, old_view(old, s), s.scores, 16, 4, pos, s.ews, s.dev_err)
    assert fg.fastgen_read_error(s.dev_err) == fg.FG_EINVAL
    for x, y in zip(before, (s.cache.k_pages, s.cache.rows, s.cache.page_table, s.scores)):
        assert torch.equal(x, y)
    q2 = dev(torch.randn(8, d, generator=g).to(torch.bfloat16))
    kv = [dev(torch.randn(8, d, generator=g).to(torch.bfloat16)) for _ in range(2)]
    got = f.decode(q2, *kv, dev([5, 6], torch.int32), n)
    assert fg.fastgen_read_error(f.dev_err) == fg.FG_EINVAL and torch.isfinite(got).all()


def old_view(old, s):
    """The retired cache's descriptors and counts with the new cache's pages."""
    c = s.cache
    return fg.PagedCache(s.p, c.k_pages, c.v_pages, c.exps, c.pos, old.page_table, old.caches,
                         old.rows, c.next_page)
