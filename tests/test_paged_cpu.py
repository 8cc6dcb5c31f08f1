"""The rotation and the paged calls without a GPU: sizes, the rotation table
and every refusal on the host, before anything is launched."""
import ctypes
import math
import os
import random

import pytest
import torch

from adaptive_head_kv_gb300 import fastgen as fg

FAKE = 1 << 20  # an aligned address never dereferenced: checks fail first


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(fg.LIB_PATH):
        from adaptive_head_kv_gb300.build import build

        build()
    fg.lib()


def P(**kw):
    base = dict(B=2, L=2, H=4, n=100, d=128, dtype=fg.FG_BF16, T=0.95, r_l=0.3, r_f=0.3, scale=0.0,
                Hkv=2)
    base.update(kw)
    return fg.Params(**base)


def cache(p, **kw):
    c = fg.PagedCacheStruct()
    for name in ("k_pages", "v_pages", "exps", "pos", "page_table", "caches", "rows", "rows_out",
                 "next_page", "sched"):
        setattr(c, name, FAKE)
    c.table_len = 100
    c.sched_bytes = fg.fastgen_paged_sched_bytes(p, 100)
    c.n_pages, c.n_work, c.n_ctas = 50, 40, 30
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rope(**kw):
    r = fg.RopeStruct(FAKE, 128, fg.FG_ROPE_HALF)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def test_struct_sizes():
    assert ctypes.sizeof(fg.RopeStruct) == 16
    assert ctypes.sizeof(fg.PagedDesc) == 24
    assert ctypes.sizeof(fg.PagedCacheStruct) == 104
    assert ctypes.sizeof(fg.PagedInfo) == 12


def test_sizes():
    al = lambda x: (x + 255) // 256 * 256
    p = P()  # 8 caches, window 30
    assert fg.fastgen_paged_table_len(p, 28) == 8 * (2 + 1)
    assert fg.fastgen_paged_table_len(p, 29) == 8 * (3 + 1)
    assert fg.fastgen_paged_table_len(P(r_l=0.0), 0) == 8 * 2
    assert fg.fastgen_paged_table_len(p, -1) == 0 and fg.fastgen_paged_table_len(P(d=96), 1) == 0
    assert fg.fastgen_paged_table_len(P(B=4000, L=100, n=100000), 100000) == 0  # past 2^31
    assert fg.fastgen_paged_sched_bytes(p, 24) == (256 + al(8 * 16) + al((24 // 4 + 17) * 24)
                                                     + (24 // 4 + 18) * 4)
    assert fg.fastgen_paged_sched_bytes(p, 0) == 0
    assert fg.fastgen_append_q8_workspace_bytes(p, 5) == (al(2 * 2 * 5 * 4) + al(8 * 2 * 4)
                                                          + al(2 * 5 * 64 * 8))
    for m in (0, -1, (1 << 20) + 1):
        assert fg.fastgen_append_q8_workspace_bytes(p, m) == 0
    size = fg.lib().fastgen_decode_q8_workspace_bytes
    assert size(p, cache(p, n_work=13)) == al(13 * 2 * 8) + al(13 * 2 * 128 * 4)
    assert size(p, cache(p, n_work=-1)) == 0


def test_rope_table():
    """turns = inv_freq / 2 pi modulo one turn, to 2^-53 relative, as 64-bit fractions."""
    rng = random.Random(1)
    f = [1.0, 1e-4, 0.0, 6.283185307179586, 7.5] + [rng.uniform(0, 1) for _ in range(50)]
    got = [int(x) % (1 << 64) for x in fg.fastgen_rope_table(f).tolist()]
    for x, t in zip(f, got):
        turn = x / (2 * math.pi)
        want = (turn - math.floor(turn)) * 2.0 ** 64
        off = abs(t - want)
        assert min(off, 2.0 ** 64 - off) <= 1 + 2.0 ** 64 * 2.0 ** -52 * max(turn, 1.0)
    for bad in ([-1.0], [float("nan")], [float("inf")], []):
        with pytest.raises(fg.FastGenError):
            fg.fastgen_rope_table(bad)


def test_rope_rejects_on_host():
    def call(p=None, Q=FAKE, K=FAKE, pos=FAKE, r=None, Qo=FAKE, Ko=FAKE):
        return fg.lib().fastgen_rope(p or P(), Q, K, pos, r or rope(), Qo, Ko, None)

    assert call(p=P(d=96)) == fg.FG_EDTYPE and call(p=P(n=0)) == fg.FG_EINVAL
    for kw in (dict(Q=None), dict(Ko=None), dict(Q=FAKE + 8), dict(Ko=FAKE + 2), dict(pos=FAKE + 2),
               dict(Q=None, K=None, Qo=None, Ko=None), dict(r=rope(turns=None)),
               dict(r=rope(turns=FAKE + 4)), dict(r=rope(rot_dim=0)), dict(r=rope(rot_dim=24)),
               dict(r=rope(rot_dim=144)), dict(r=rope(style=2)), dict(p=P(d=64))):
        assert call(**kw) == fg.FG_EINVAL, kw
    assert fg.lib().fastgen_rope(P(), FAKE, FAKE, None, None, FAKE, FAKE, None) == fg.FG_EINVAL


LAYOUT = [dict(page_table=None), dict(caches=None), dict(rows=None), dict(table_len=0),
          dict(caches=FAKE + 4), dict(page_table=FAKE + 1), dict(rows=FAKE + 2)]
PAGES = [dict(k_pages=None), dict(v_pages=None), dict(exps=None), dict(pos=None), dict(n_pages=0),
         dict(k_pages=FAKE + 8), dict(v_pages=FAKE + 8), dict(exps=FAKE + 4), dict(pos=FAKE + 8)]


def test_plan_and_schedule_reject_on_host():
    L, p, info = fg.lib(), P(), fg.PagedInfo()

    def plan(p=p, policy=FAKE, keep=FAKE, new=28, out=info, **kw):
        return L.fastgen_paged_plan(p, policy, keep, new, cache(P(), **kw), out, None)

    for kw in LAYOUT + [dict(next_page=None), dict(next_page=FAKE + 2), dict(sched=None),
                        dict(sched=FAKE + 64), dict(policy=None), dict(keep=None), dict(new=-1),
                        dict(out=None), dict(p=P(T=0.0))]:
        assert plan(**kw) == fg.FG_EINVAL, kw
    assert plan(p=P(d=32)) == fg.FG_EDTYPE
    assert plan(table_len=23) == fg.FG_EWORKSPACE
    assert plan(sched_bytes=cache(p).sched_bytes - 1) == fg.FG_EWORKSPACE
    assert plan(sched_bytes=-1) == fg.FG_EWORKSPACE
    assert L.fastgen_paged_plan(p, FAKE, FAKE, 4, None, info, None) == fg.FG_EINVAL
    for kw in LAYOUT + [dict(sched=None), dict(sched=FAKE + 64)]:
        assert L.fastgen_paged_schedule(p, cache(p, **kw), None) == fg.FG_EINVAL, kw
    assert L.fastgen_paged_schedule(p, cache(p, sched_bytes=0), None) == fg.FG_EWORKSPACE


def test_compact_rejects_on_host():
    L, p = fg.lib(), P()

    def call(p=p, K=FAKE, V=FAKE, keep=FAKE, err=FAKE, **kw):
        return L.fastgen_compact_q8(p, K, V, keep, cache(P(), **kw), err, None)

    for kw in LAYOUT + PAGES + [dict(K=None), dict(V=FAKE + 8), dict(keep=None), dict(err=None),
                                dict(err=FAKE + 1), dict(p=P(H=5))]:
        assert call(**kw) == fg.FG_EINVAL, kw
    assert call(p=P(dtype=3)) == fg.FG_EDTYPE


def test_append_rejects_on_host():
    L, p = fg.lib(), P()
    need = fg.fastgen_append_q8_workspace_bytes(p, 5)

    def call(p=p, k=FAKE, v=FAKE, ids=FAKE, m=5, n_new=FAKE, ns=1, sp=FAKE, np_=1, at=FAKE,
             r=None, ws=FAKE, ws_bytes=need, err=FAKE, **kw):
        return L.fastgen_append_q8(p, cache(P(), **kw), k, v, ids, m, n_new, sp, ns, FAKE, np_, at,
                                   r or rope(), ws, ws_bytes, err, None)

    for kw in LAYOUT + PAGES + [
            dict(next_page=None), dict(next_page=FAKE + 1), dict(rows_out=FAKE + 1), dict(k=None),
            dict(v=None), dict(k=FAKE + 8), dict(ids=None), dict(ids=FAKE + 2), dict(m=0),
            dict(m=(1 << 20) + 1), dict(n_new=FAKE + 2), dict(ns=-1), dict(sp=None),
            dict(np_=5000), dict(at=None), dict(at=FAKE + 2), dict(r=rope(rot_dim=8)),
            dict(r=rope(style=-1)), dict(ws=None), dict(ws=FAKE + 128), dict(err=None)]:
        assert call(**kw) == fg.FG_EINVAL, kw
    assert call(ws_bytes=need - 1) == fg.FG_EWORKSPACE
    assert call(p=P(d=80)) == fg.FG_EDTYPE
    assert call(p=P(B=70000, L=1, H=1, Hkv=1)) == fg.FG_EINVAL


def test_decode_rejects_on_host():
    L, p = fg.lib(), P()
    need = fg.lib().fastgen_decode_q8_workspace_bytes(p, cache(p))

    def call(p=p, q=FAKE, k=FAKE, v=FAKE, ids=FAKE, ns=1, at=FAKE, r=None, out=FAKE, ws=FAKE,
             ws_bytes=need, err=FAKE, **kw):
        return L.fastgen_decode_attn_q8(p, cache(P(), **kw), q, k, v, ids, FAKE, ns, FAKE, 1, at,
                                        r or rope(), out, ws, ws_bytes, err, None)

    for kw in LAYOUT + PAGES + [
            dict(sched=None), dict(sched=FAKE + 32), dict(n_work=0), dict(n_work=7),
            dict(n_work=1 << 20), dict(n_ctas=0), dict(n_ctas=41),
            dict(next_page=None), dict(q=None), dict(q=FAKE + 8), dict(k=None), dict(v=None),
            dict(v=FAKE + 8), dict(ids=None), dict(ns=9999), dict(at=None), dict(out=None),
            dict(out=FAKE + 4), dict(ws=None), dict(ws=FAKE + 16), dict(err=None),
            dict(r=rope(rot_dim=256)), dict(rows_out=FAKE + 3)]:
        assert call(**kw) == fg.FG_EINVAL, kw
    assert call(ws_bytes=need - 1) == fg.FG_EWORKSPACE
    assert call(sched_bytes=10) == fg.FG_EWORKSPACE
    assert call(p=P(dtype=2)) == fg.FG_EDTYPE
    # without a new token neither ids nor a page counter are needed: refused for the workspace only
    assert call(k=None, v=None, ids=None, next_page=None, ws_bytes=0) == fg.FG_EWORKSPACE


def test_binding_refuses_tensors_that_do_not_fit():
    """Types, sizes and devices are checked before the library is called."""
    p = P(B=1, L=1, H=2, Hkv=2, n=10)
    i32 = dict(dtype=torch.int32)
    parts = dict(page_table=torch.zeros(8, **i32), caches=torch.zeros(2, 6, **i32),
                 rows=torch.zeros(2, **i32), next_page=torch.zeros(1, **i32))
    pages = dict(k_pages=torch.zeros(3, 64, 128, dtype=torch.uint8),
                 v_pages=torch.zeros(3, 64, 128, dtype=torch.uint8),
                 exps=torch.zeros(3, 4, 2, dtype=torch.int8), pos=torch.zeros(3, 64, **i32))
    make = lambda **kw: fg.PagedCache(p, **{**pages, **parts, **kw})
    c = make()
    assert c.c.n_pages == 3 and c.c.table_len == 8
    for kw in (dict(caches=torch.zeros(2, 5, **i32)), dict(rows=torch.zeros(2)),
               dict(rows=torch.zeros(3, **i32)), dict(rows_out=torch.zeros(1, **i32)),
               dict(k_pages=torch.zeros(2, 64, 128, dtype=torch.uint8)),
               dict(v_pages=torch.zeros(3, 64, 128)), dict(pos=torch.zeros(64, 3, **i32).t())):
        with pytest.raises(fg.FastGenError) as e:
            make(**kw)
        assert e.value.status == fg.FG_EINVAL
    rp = fg.Rope.make(128, device="cpu")
    assert rp.c.rot_dim == 128
    err, pos = torch.zeros(1, **i32), torch.zeros(1, **i32)
    kv = torch.zeros(2, 128, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    bad = [lambda: fg.Rope(torch.zeros(64)),
           lambda: fg.fastgen_rope(p, kv, kv, None, rp, kv, kv),
           lambda: fg.fastgen_rope(p, None, None, None, rp, None, None),
           lambda: fg.fastgen_compact_q8(p, kv, kv, kv, c, err),
           lambda: fg.fastgen_append_q8(p, c, kv.float(), kv, pos, None, None, None, pos, rp, ws, err),
           lambda: fg.fastgen_append_q8(p, c, kv, kv, torch.zeros(2, **i32), None, None, None, pos,
                                        rp, ws, err),
           lambda: fg.fastgen_decode_attn_q8(p, c, kv, kv, kv, pos.long(), None, None, pos, rp, kv,
                                             ws, err),
           lambda: fg.fastgen_decode_attn_q8(P(B=1, L=1, H=2, Hkv=2, n=10, d=64), c, kv[:, :64].contiguous(),
                                             None, None, None, None, None, pos, None,
                                             kv[:, :64].contiguous(), ws, err),
           # sizes fit, but nothing runs on the CPU
           lambda: fg.fastgen_decode_attn_q8(p, c, kv, kv, kv, pos, None, None, pos, rp, kv, ws, err)]
    for call in bad:
        with pytest.raises(fg.FastGenError) as e:
            call()
        assert e.value.status == fg.FG_EINVAL
