"""How near the paged 8-bit calls come to their definition, with bounds that
leave no room for operands of fewer bits."""
import numpy as np
import pytest
import torch

import paged_ref as P
import test_paged_gpu as T
from adaptive_head_kv_gb300 import fastgen as fg

pytestmark = pytest.mark.gpu


def pair_sizes(q, rot, half):
    """|x| + |y| of the pair that each rotated value belongs to (0 where nothing is rotated)."""
    a, out = np.abs(q), np.zeros_like(q)
    i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if half
            else (slice(0, rot, 2), slice(1, rot, 2)))
    out[i] = out[j] = a[i] + a[j]
    return out


def near(q, k, v, ev, scale, dtype, pair):
    """(output, how far it may be off) of one query, for either type: queries and weights enter
    the products with 22 bits (2^-21 of each covers both f16 terms), products are summed in 32
    bits (2^-20 of the sum of magnitudes), a rotated value is off by 2^-21 of its pair's size (cos,
    sin, two products and a sum in 32 bits), exponentials and sums add 2^-19, and only the result
    is rounded to its type (bf16 2^-8, fp32 2^-24).  A score off by ds changes each weight by a
    factor within e^(+-2 ds)."""
    want, weight, products, floor = P.attend(q, k, v, ev, scale)
    turned = scale * float((np.abs(k) @ pair).max()) if len(k) else 0.0
    ds = products * (2.0 ** -21 + 2.0 ** -20) + turned * 2.0 ** -21
    rel = np.expm1(2 * ds) + 2.0 ** -20 + 2.0 ** -19
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return want, rel * weight + floor * (1 + rel) + half * np.abs(want) + 1e-30


def check_near(s, out, q, pos, rot=0, half=False, inv=None):
    got = T.f64(out)
    for g in range(s.G):
        hkv = s.p.Hkv or s.p.H
        c = (g // s.p.H) * hkv + (g % s.p.H) // s.R
        qq = T.f64(q[g])
        pair = pair_sizes(qq, rot, half)
        if rot:
            qq = P.rotate(qq, pos[c // s.hl], inv, half)
        k, v, ev = s.ref[c].kv(pos[c // s.hl])
        want, bound = near(qq, k, v, ev, 1 / np.sqrt(s.d), s.dtype, pair)
        off = np.abs(got[g] - want)
        assert (off <= bound).all(), (g, (off / bound).max(), len(k))


@pytest.mark.parametrize("rot,half", [(0, False), (64, False), (64, True)])
@pytest.mark.parametrize("kw", [dict(n=400), dict(n=400, d=64), dict(H=8, Hkv=2, n=333),
                                dict(H=8, Hkv=2, n=150, d=64), dict(n=400, dtype="fp32"),
                                dict(H=16, Hkv=2, n=333, d=64, dtype="fp32"), dict(n=1500, L=1)])
def test_decode_rounds_nothing_but_its_result(kw, rot, half):
    """Queries, weights and sums keep 22 bits and more, in both types (but for bf16 groups of 8)."""
    s = T.Setup(40, **kw)
    s.compact()
    inv, turns = T.table(rot) if rot else (None, None)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED) if rot else None
    for i, at in enumerate((s.n - 1, s.n + 70000)):  # all rows; without the ring's
        q = torch.randn(s.G, s.d, generator=T.gen(i)).to(T.DT[s.dtype])
        out = s.decode(q, None, None, None, [at], rope)
        check_near(s, out, q, [at], rot, half, inv)
    assert int(s.err.item()) == 0


@pytest.mark.parametrize("kw,order", [(kw, order) for order in ("first", "last", "turns") for kw in (
    dict(H=2, n=160), dict(H=8, Hkv=2, n=240, d=64), dict(H=8, Hkv=1, n=1300))]
    + [(dict(B=16, L=8, H=8, n=130, r_l=0.0), "turns")])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_of_zero_beside_large_ones_keep_their_weight(kw, order, dtype):
    """Blocks of zero values have the least exponent; their rows hold half the attention all the
    same, in one item, in several and in shared thread blocks."""
    def plant(s):
        block = torch.arange(s.n) // 16
        half = s.n // 32
        zero = {"first": block < half, "last": block >= half, "turns": block % 2 == 0}[order]
        s.V[:] = (s.V.float() * size).to(s.V.dtype)
        s.V[:, zero] = 0
        s.V[:, ~zero, 1] = size
        s.K[:, zero] *= 1.25
    for size in (2.0 ** 36, 2.0 ** 100) if "B" not in kw else (2.0 ** 60,):
        s = T.Setup(41, dtype=dtype, policies=[4], plant=plant, **{"L": 1, **kw})
        s.compact()
        q = torch.randn(s.G, s.d, generator=T.gen(1)).to(T.DT[dtype])
        out = s.decode(q, None, None, None, [s.n - 1] * s.B)
        s.check_out(out, q, [s.n - 1] * s.B)
        assert int(s.err.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [192, 2600])
def test_small_weights_meet_large_values(n, dtype):
    """Rows of weight 2^-100 and less whose values outweigh all others, in one item and across
    items."""
    def plant(s):
        s.K[:] = 0
        s.V[:] = (s.V.float() * 2.0 ** -60).to(s.V.dtype)
        s.K[:, -32:, 0] = -16.0
        s.V[:, -32:] = (torch.rand(s.gk, 32, s.d, generator=T.gen(5)) + 0.5).to(s.V.dtype) * 2.0 ** 60
    s = T.Setup(42, L=1, H=2, n=n, dtype=dtype, policies=[4], plant=plant)
    s.compact()
    for first in (4.0, 50.0, 80.0, 110.0):
        q = torch.zeros(s.G, s.d)
        q[:, 0] = first
        q = q.to(T.DT[dtype])
        out = s.decode(q, None, None, None, [n - 1])
        s.check_out(out, q, [n - 1])
    assert int(s.err.item()) == 0
