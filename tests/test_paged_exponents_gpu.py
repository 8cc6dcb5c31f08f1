"""Exponents that are nobody's, or as small as they get: a block of 16 rows without a row has
whatever byte its memory held, and a block of zeros the least exponent there is.  Neither may reach
a result."""
import pytest
import torch

import paged_ref as P
from adaptive_head_kv_gb300 import fastgen as fg
from test_paged_gpu import DT, Setup, dev, gen
from test_paged_step_gpu import Fork, Step, check_cut

pytestmark = pytest.mark.gpu

FILLS = [-128, -127, -100, 127]


class Filled:
    """Page pools whose exponents hold `byte` before anything is coded."""

    byte = 17

    def set_pages(self, count):
        super().set_pages(count)
        self.cache.exps.fill_(self.byte)


def filled(kind, byte):
    return type(kind.__name__, (Filled, kind), dict(byte=byte))


def queries(f, seed):
    """Of three heads one of zeros, one far below what f16 holds, one as usual."""
    q = torch.randn(f.G, f.d, generator=gen(seed))
    q[::3] = 0.0
    q[1::3] *= 2.0 ** -40
    return q.to(DT[f.dtype])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("fp32", 128), ("fp32", 64)])
@pytest.mark.parametrize("B,H,Hkv", [(3, 2, 2), (5, 8, 2), (150, 2, 2)])
@pytest.mark.parametrize("n", [1, 16, 17, 48, 63, 113])
def test_blocks_without_a_row_behind_a_prompt(n, B, H, Hkv, dtype, d):
    """A prompt whose segments and rings end inside a page: every remainder of rows, one and
    two tiles of queries, before and after the sequences have rows of their own."""
    first = None
    for byte in [17] + FILLS:
        s = filled(Setup, byte)(50, B=1, L=1, H=H, Hkv=Hkv, n=n, d=d, dtype=dtype, max_new=1,
                                policies=[4] * (H // Hkv) + [3] * (H // Hkv))
        s.compact()
        f = filled(Fork, byte)(s, B)
        outs = []
        for st in range(2):
            pos = [n + st + b % 3 for b in range(B)]
            q = queries(f, st)
            ids, k, v = f.tokens(st, 1) if st else (None, None, None)
            outs.append(f.decode(q, ids, k, v, pos))
            if first is None:
                if st:
                    f.ref_append(ids, k, v, pos)
                f.check_out(outs[-1], q, pos)
        if first is None:
            first = outs
        for x, y in zip(first, outs):
            assert torch.equal(x, y), byte
        assert int(f.err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [2, 150])
def test_zeros_meet_zeros_behind_a_prompt(B, dtype):
    """Queries of zeros, and small ones, over blocks of zero keys beside rows that are not there, and
    over ring blocks without a position, or with positions that left the window."""
    def segment(s):  # rows 16-19 of a page
        s.K[:, 16:] = 0.0

    def ring(s):  # slots 16 and 17 of 18, of tokens that went to the segment
        s.keep[:, 52:54] = 1
        s.K[:, 39:45] = 0.0

    for n, policy, plant in ((20, 4, segment), (57, 3, ring)):
        s = Setup(51, B=1, L=1, H=2, n=n, dtype=dtype, max_new=1, policies=[policy], plant=plant)
        s.compact()
        f = Fork(s, B)
        e = P.GpuPages(s.cache).segment(0, policy == 3, 18 if policy == 3 else 20)["ek"]
        assert e[1] == P.E_MIN
        for q in (queries(f, 1), torch.zeros(f.G, f.d, dtype=DT[dtype]),
                  (torch.randn(f.G, f.d, generator=gen(2)) * 2.0 ** -90).to(DT[dtype])):
            for pos in ([n + b % 3 for b in range(B)], [n + 10 + b % 20 for b in range(B)],
                        [n if b % 2 else -1 for b in range(B)]):
                f.check_out(f.decode(q, None, None, None, pos), q, pos)
        assert int(f.err.item()) == 0


@pytest.mark.parametrize("byte", FILLS)
@pytest.mark.parametrize("B,kw", [(3, dict(H=8, Hkv=1, n=81)), (4, dict(H=8, Hkv=2, n=70, d=64)),
                                  (5, dict(n=49, dtype="fp32")), (16, dict(n=90, L=8, H=8))])
def test_weights_and_small_caches_behind_a_prompt(B, kw, byte):
    s = filled(Setup, byte)(52, B=1, max_new=1, **kw)
    s.compact()
    f = filled(Fork, byte)(s, B, 12).with_scores(1)
    for st in range(3):
        pos = [f.n + st + b % 4 if (st + b) % 4 else -1 for b in range(B)]
        f.step(st, pos, scale=(1, 0, 2.0 ** -40)[st], check=st == 2)
    assert int(f.err.item()) == 0


@pytest.mark.parametrize("byte", FILLS)
@pytest.mark.parametrize("kw", [dict(), dict(H=8, Hkv=1, n=113), dict(d=64, n=77, dtype="fp32")])
def test_steps_appends_and_cuts(kw, byte):
    """Without a prompt: the plain step, the step that keeps weights, appended rows, the cut."""
    a, s = filled(Setup, byte)(53, **kw), filled(Step, byte)(53, **kw)
    a.compact()
    s.compact()
    s.with_scores(1)
    for st in range(3):
        ids, k, v = a.tokens(st, 1)
        q = queries(a, st)
        a.check_out(a.decode(q, None, None, None, [a.n + 2 * st]), q, [a.n + 2 * st])
        a.append(*a.tokens(9 + st, 2), [a.n + 2 * st])
        a.ref_append(*a.tokens(9 + st, 2), [a.n + 2 * st])
        a.check()
        s.step(st, [s.n + st], scale=(1, 0, 2.0 ** -40)[st])
    assert check_cut(s, 32, 5, [s.n + 2]) > 0
    s.check()
    assert int(a.err.item()) == 0 and int(s.err.item()) == 0
