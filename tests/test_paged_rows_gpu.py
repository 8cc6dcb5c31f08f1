"""Decode steps on long caches, with every row in the outputs: work lists cut
in lengths, long items, idle sequences, lists made anew."""
import numpy as np
import pytest
import torch

import paged_count as C
import paged_ref as P
import test_paged_gpu as T

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def only_positions(monkeypatch):
    monkeypatch.setattr(P, "RefCache", C.Positions)


class Setup(T.Setup):
    def __init__(self, seed, step, **kw):
        self.step = step

        def plant(s):
            s.V[:] = C.values(np.arange(s.n), s.d, step).to(s.V.dtype)
        super().__init__(seed, plant=plant, **kw)
        self.q = torch.zeros(self.G, self.d, dtype=T.DT[self.dtype])

    def turn(self, seed, m, pos):
        """Tokens at pos (a list) with their positions' values."""
        ids, k, v = self.tokens(seed, m)
        for c in range(self.gk):
            at = max(pos[c // self.hl], 0) + np.arange(m)
            v[c] = C.values(at, self.d, self.step).to(v.dtype)
        return ids, k, v

    def check_out(self, out, pos):
        got = T.f64(out)
        hkv = self.p.Hkv or self.p.H
        for c, r in enumerate(self.ref):
            b = c // self.hl
            g0 = (c // hkv) * self.p.H + (c % hkv) * self.R
            mine = got[g0: g0 + self.R]
            if pos[b] < 0:
                assert (mine == 3.5).all()
                continue
            want = C.counts(r.positions(pos[b]), self.d, self.step)
            assert (np.abs(mine - want) <= C.bound(want, self.dtype)).all(), (
                c, r.rows, np.abs(mine - want).max())


@pytest.mark.parametrize("step", [0, 1])
@pytest.mark.parametrize("kw", [
    dict(n=1300, L=1, r_l=0.45), dict(n=2600, L=1, H=4, Hkv=1), dict(n=2600, L=1, dtype="fp32"),
    dict(n=4200, L=1, H=8, Hkv=1, d=64), dict(n=4200, L=2, H=16, Hkv=4, dtype="fp32"),
    dict(n=700, L=1, H=8, Hkv=1, dtype="fp32", d=64), dict(B=2, L=16, H=32, n=70, d=64),
    dict(B=3, L=10, H=64, Hkv=32, n=50), dict(n=200, L=1), dict(n=1, L=1)])
def test_steps(kw, step):
    s = Setup(60, step, max_new=200, **kw)
    s.compact()
    at = s.n
    for i in range(4):
        pos = [at + 3 * b for b in range(s.B)]
        ids, k, v = s.turn(i, 1, pos)
        out = s.decode(s.q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
        s.check_out(out, pos)
        at += 1
        if i == 1:  # a turn of several tokens, and the list made anew
            for m in (7, 70):
                pos = [at + 3 * b for b in range(s.B)]
                ids, k, v = s.turn(20 + m, m, pos)
                s.append(ids, k, v, pos)
                s.ref_append(ids, k, v, pos)
                at += m
            out = s.decode(s.q, None, None, None, [p + m - 1 for p in pos])
            s.check_out(out, [p + m - 1 for p in pos])
            s.cache.schedule(s.p)
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kw,idle", [
    (dict(B=4, L=4, H=8, n=2600, d=64, policies=[4, 4, 3, 4]), [[0], [3], [1, 2], [0, 1, 2], []]),
    (dict(B=40, L=3, H=8, n=70), [[0, 5, 31, 32, 39], range(1, 40), range(39), [7], range(40)]),
    (dict(B=2, L=2, H=64, Hkv=32, n=4200, policies=[4, 3, 1, 2]), [[0], [1]]),
    (dict(B=2, L=2, H=64, Hkv=16, n=4200, policies=[4, 3, 4, 1]), [[0], [1]]),
    (dict(B=2, L=2, H=64, Hkv=8, n=4200, policies=[4] * 8 + [3] * 8), [[0], [1], []])])
def test_idle_sequences_of_lists_of_equal_lengths(kw, idle, dtype):
    s = Setup(61, 1, max_new=8, dtype=dtype, **kw)
    if s.R < 8:
        assert int(s.cache.sched.view(torch.int32)[64 + 3]) > 0  # a list of equal lengths
    s.compact()
    now = np.full(s.B, s.n)
    for st, off in enumerate(idle):
        pos = [-1 if b in off else int(now[b]) for b in range(s.B)]
        ids, k, v = s.turn(st, 1, pos)
        out = s.decode(s.q, ids, k, v, pos)
        s.ref_append(ids, k, v, pos)
        s.check_out(out, pos)
        now += [p >= 0 for p in pos]
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype,d,H", [("bf16", 128, 8), ("fp32", 128, 8), ("bf16", 64, 16)])
def test_items_that_grew_by_thousands_of_rows(dtype, d, H):
    s = Setup(62, 1, L=1, H=H, Hkv=2, n=30, d=d, dtype=dtype, max_new=5000, r_l=0.9,
              policies=[4] * (H // 2) + [3] * (H // 2))
    s.compact()
    at = 30
    for m in (2500, 33, 32, 1):
        ids, k, v = s.turn(m, m, [at])
        s.append(ids, k, v, [at])
        s.ref_append(ids, k, v, [at])
        at += m
        s.check_out(s.decode(s.q, None, None, None, [at - 1]), [at - 1])
    s.cache.schedule(s.p)
    s.check_out(s.decode(s.q, None, None, None, [at - 1]), [at - 1])
    ids, k, v = s.turn(1, 1, [at])
    out = s.decode(s.q, ids, k, v, [at])
    s.ref_append(ids, k, v, [at])
    s.check_out(out, [at])
    assert int(s.err.item()) == 0
