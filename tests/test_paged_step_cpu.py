"""Steps behind a shared prompt, the rows' weights and the cut to a budget without a GPU: sizes,
and every refusal on the host, before anything is launched."""
import pytest
import torch

import test_paged_cpu as C
from adaptive_head_kv_gb300 import fastgen as fg
from adaptive_head_kv_gb300.session import PagedSession, make_params
from test_paged_cpu import FAKE, LAYOUT, P, PAGES, built, cache, rope  # noqa: F401

al = lambda x: (x + 255) // 256 * 256
OTHER = FAKE + 4096
PREFIX = dict(caches=OTHER, rows=OTHER, page_table=OTHER)  # not the ones that a step appends to


def test_fork_table_len():
    p = P()  # 8 caches, window 30
    assert fg.fastgen_paged_fork_table_len(p, 64) == 8 * (1 + 1)
    assert fg.fastgen_paged_fork_table_len(p, 65) == 8 * (2 + 1)
    assert fg.fastgen_paged_fork_table_len(p, 0) == 8 * (1 + 1)
    assert fg.fastgen_paged_fork_table_len(P(r_l=0.0), 1000) == 8 * 16
    assert fg.fastgen_paged_fork_table_len(p, -1) == 0
    assert fg.fastgen_paged_fork_table_len(P(d=96), 10) == 0
    assert fg.fastgen_paged_fork_table_len(p, 2 ** 31 - 1) == 0
    assert fg.fastgen_paged_fork_table_len(P(B=5000, L=100), 2 ** 20) == 0  # past 2^31


@pytest.mark.parametrize("dtype,B,Hkv,d", [(fg.FG_BF16, 2, 2, 128), (fg.FG_FP32, 2, 2, 128),
                                           (fg.FG_BF16, 90, 2, 64), (fg.FG_FP32, 200, 1, 64)])
def test_workspace_bytes(dtype, B, Hkv, d):
    """Own partial results, the pool's scores, the heads' sums, then what the shared caches take:
    counts, queries in tiles of 128, factors, two partial results for 192 thread blocks and every
    group of one cache's queries."""
    p, R = P(dtype=dtype, B=B, Hkv=Hkv, d=d), 4 // Hkv
    c = cache(p, n_work=13)
    own = al(13 * R * 8) + al(13 * R * d * 4)
    size = lambda pre, sc: fg.lib().fastgen_decode_q8_ex_workspace_bytes(p, c, c if pre else None, sc)
    assert size(False, 0) == own
    scores = al(50 * 64 * R * 4) + al(B * 2 * 4 * 8)
    assert size(False, 1) == own + scores
    caches, nq = 2 * Hkv, B * R
    tiles, terms = -(-nq // 128), 1 if dtype == fg.FG_BF16 else 2
    groups = -(-tiles // 2) if terms == 1 and tiles > 1 else tiles
    parts = 2 * (192 + caches * groups) * min(nq, 128)
    shared = (al((caches + 1) * 8) + al(caches * tiles * terms * 128 * d * 2)
              + al(caches * tiles * 128 * 4) + al(parts * 8) + al(parts * d * 4))
    assert size(True, 0) == own + shared
    assert size(True, 7) == own + scores + shared
    assert fg.lib().fastgen_decode_q8_ex_workspace_bytes(p, cache(p, n_work=-1), None, 0) == 0
    assert fg.lib().fastgen_decode_q8_ex_workspace_bytes(P(d=32), c, None, 0) == 0


def test_evict_workspace_bytes():
    p = P()  # 8 caches
    assert fg.fastgen_evict_q8_workspace_bytes(p, 48) == al(8 * 4) + al(8 * 48 * 8)
    for budget in (0, -16, 17, 8):
        assert fg.fastgen_evict_q8_workspace_bytes(p, budget) == 0
    assert fg.fastgen_evict_q8_workspace_bytes(P(B=0), 16) == 0


def test_step_rejects_on_host():
    L, p = fg.lib(), P()
    need = L.fastgen_decode_q8_ex_workspace_bytes(p, cache(p), cache(p), 1)

    def call(p=p, q=FAKE, k=FAKE, v=FAKE, ids=FAKE, ns=1, at=FAKE, r=None, out=FAKE, ws=FAKE,
             ws_bytes=need, err=FAKE, scores=FAKE, prefix=None, **kw):
        shared = cache(P(B=1), **{**PREFIX, **(prefix or {})})
        return L.fastgen_decode_attn_q8_ex(p, cache(P(), **kw), shared, scores, q, k, v, ids, FAKE,
                                           ns, FAKE, 1, at, r or rope(), out, ws, ws_bytes, err,
                                           None)

    assert call(ws_bytes=0) == fg.FG_EWORKSPACE  # nothing else is wrong
    for kw in LAYOUT + PAGES + [dict(prefix=x) for x in LAYOUT + PAGES] + [
            dict(sched=None), dict(sched=FAKE + 32), dict(n_work=0), dict(n_work=7),
            dict(n_work=1 << 20), dict(n_ctas=0), dict(n_ctas=41), dict(next_page=None),
            dict(q=None), dict(q=FAKE + 8), dict(k=None), dict(v=None), dict(v=FAKE + 8),
            dict(ids=None), dict(ns=9999), dict(at=None), dict(at=FAKE + 2), dict(out=None),
            dict(out=FAKE + 4), dict(ws=None), dict(ws=FAKE + 16), dict(err=None),
            dict(prefix=dict(caches=FAKE)), dict(prefix=dict(rows=FAKE)),
            dict(prefix=dict(page_table=FAKE)),
            dict(scores=FAKE + 4), dict(r=rope(rot_dim=256)), dict(rows_out=FAKE + 3)]:
        assert call(**kw) == fg.FG_EINVAL, kw
    assert call(ws_bytes=need - 1) == fg.FG_EWORKSPACE
    assert call(sched_bytes=10) == fg.FG_EWORKSPACE
    assert call(p=P(dtype=2)) == fg.FG_EDTYPE
    # a prefix's list, counter and counts out are not used
    assert call(prefix=dict(sched=None, next_page=None, rows_out=None, n_work=0),
                ws_bytes=0) == fg.FG_EWORKSPACE
    # without options: refused for the workspace only
    assert L.fastgen_decode_attn_q8_ex(p, cache(p), None, None, FAKE, None, None, None, None, 0, None,
                                       0, FAKE, None, FAKE, FAKE, 0, FAKE, None) == fg.FG_EWORKSPACE


def test_fork_and_clear_reject_on_host():
    L, p, info = fg.lib(), P(), fg.PagedInfo()

    def fork(p=p, new=64, out=info, prefix=None, **kw):
        return L.fastgen_paged_fork(p, cache(P(B=1), **{**PREFIX, **(prefix or {})}), new,
                                    cache(P(), **kw), out, None)

    for kw in LAYOUT + [dict(next_page=None), dict(next_page=FAKE + 2), dict(sched=None),
                        dict(sched=FAKE + 64), dict(new=-1), dict(out=None), dict(p=P(T=0.0)),
                        dict(prefix=dict(caches=FAKE)), dict(prefix=dict(caches=None)), dict(prefix=dict(caches=FAKE + 4))]:
        assert fork(**kw) == fg.FG_EINVAL, kw
    assert fork(table_len=15) == fg.FG_EWORKSPACE
    assert fork(sched_bytes=5) == fg.FG_EWORKSPACE
    assert fork(p=P(d=32)) == fg.FG_EDTYPE
    assert L.fastgen_paged_fork(p, None, 64, cache(p), info, None) == fg.FG_EINVAL
    for kw in LAYOUT + PAGES + [dict(rows_out=FAKE + 1)]:
        assert L.fastgen_paged_clear(p, cache(p, **kw), FAKE, None) == fg.FG_EINVAL, kw
    assert L.fastgen_paged_clear(p, cache(p), None, None) == fg.FG_EINVAL
    assert L.fastgen_paged_clear(P(H=3), cache(p), FAKE, None) == fg.FG_EINVAL


def test_scores_and_evict_reject_on_host():
    L, p = fg.lib(), P()

    def scores(p=p, sc=FAKE, col=FAKE, ids=FAKE, m=5, n_new=FAKE, at=FAKE, ns=1, sp=FAKE, err=FAKE,
               **kw):
        return L.fastgen_scores_q8(p, cache(P(), **kw), sc, col, ids, m, n_new, at, sp, ns, err, None)

    for kw in LAYOUT + PAGES + [
            dict(sc=None), dict(sc=FAKE + 2), dict(col=FAKE + 1), dict(ids=None), dict(ids=FAKE + 2),
            dict(m=0), dict(n_new=FAKE + 1), dict(at=FAKE + 3), dict(ns=-1), dict(sp=None),
            dict(ns=4097), dict(err=None), dict(p=P(scale=-1.0))]:
        assert scores(**kw) == fg.FG_EINVAL, kw
    need = fg.fastgen_evict_q8_workspace_bytes(p, 48)

    def evict(p=p, sc=FAKE, budget=48, recent=48, at=FAKE, ws=FAKE, ws_bytes=need, err=FAKE, **kw):
        return L.fastgen_evict_q8(p, cache(P(), **kw), sc, budget, recent, at, ws, ws_bytes, err, None)

    for kw in LAYOUT + PAGES + [
            dict(sc=None), dict(sc=FAKE + 1), dict(budget=0), dict(budget=40), dict(budget=-16),
            dict(recent=49), dict(recent=-1), dict(at=None), dict(at=FAKE + 2), dict(ws=None),
            dict(ws=FAKE + 64), dict(err=None), dict(err=FAKE + 2), dict(rows_out=FAKE + 2)]:
        assert evict(**kw) == fg.FG_EINVAL, kw
    assert evict(ws_bytes=need - 1) == fg.FG_EWORKSPACE
    assert evict(p=P(dtype=9)) == fg.FG_EDTYPE


def test_binding_refuses_tensors_that_do_not_fit():
    i32 = dict(dtype=torch.int32)

    def make(p, pages=3):
        gk = p.B * p.L * p.Hkv
        return fg.PagedCache(p, torch.zeros(pages, 64, 128, dtype=torch.uint8),
                             torch.zeros(pages, 64, 128, dtype=torch.uint8),
                             torch.zeros(pages, 4, 2, dtype=torch.int8), torch.zeros(pages, 64, **i32),
                             torch.zeros(8, **i32), torch.zeros(gk, 6, **i32), torch.zeros(gk, **i32),
                             torch.zeros(1, **i32))

    p, one = P(B=2, L=1, H=2, Hkv=2, n=10), P(B=1, L=1, H=2, Hkv=2, n=10)
    c, pre = make(p), make(one)
    kv = torch.zeros(4, 128, dtype=torch.bfloat16)
    pos, err, ws = torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(1 << 20, dtype=torch.uint8)
    sc = torch.zeros(3, 64)
    step = lambda prefix=pre, scores=sc, q=kv: fg.fastgen_decode_attn_q8_ex(
        p, c, prefix, scores, q, kv, kv, pos, None, None, pos, None, kv, ws, err)
    bad = [step,  # everything fits, but nothing runs on the CPU
           lambda: step(prefix=c), lambda: step(prefix=make(P(B=1, L=1, H=2, Hkv=1, n=10))),
           lambda: step(scores=sc.double()), lambda: step(scores=torch.zeros(2, 64)),
           lambda: step(scores=torch.zeros(64, 3).t()), lambda: step(q=kv.float()),
           lambda: fg.fastgen_paged_fork(p, None, 10, c), lambda: fg.fastgen_paged_fork(p, c, 10, c),
           lambda: fg.fastgen_paged_clear(p, c, pos),
           lambda: fg.fastgen_scores_q8(p, c, sc, torch.zeros(4, 4), pos, None, None, None, err),
           lambda: fg.fastgen_scores_q8(p, c, torch.zeros(64), None, pos, None, None, None, err),
           lambda: fg.fastgen_evict_q8(p, c, sc, 16, 0, pos.long(), ws, err),
           lambda: fg.fastgen_evict_q8(p, c, sc, 16, 0, pos, ws.int(), err)]
    for call in bad:
        with pytest.raises(fg.FastGenError) as e:
            call()
        assert e.value.status == fg.FG_EINVAL


def test_session_refuses_budgets():
    p = make_params(1, 1, 2, 10, 64, "bf16", 0.9, 0.3, 0.3)
    for kw in (dict(budget=40), dict(budget=16, recent=17), dict(budget=16, recent=-1), dict(recent=1)):
        with pytest.raises(ValueError):
            PagedSession(p, [1], [2], 10, device="cpu", **kw)
