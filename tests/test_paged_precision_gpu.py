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


@pytest.mark.parametrize("kw,order", [(kw, order) for order in ("first", "last", "turns")
                                     for kw in (
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
        large = torch.rand(s.gk, 32, s.d, generator=T.gen(5)) + 0.5
        s.V[:, -32:] = large.to(s.V.dtype) * 2.0 ** 60
    s = T.Setup(42, L=1, H=2, n=n, dtype=dtype, policies=[4], plant=plant)
    s.compact()
    for first in (4.0, 50.0, 80.0, 110.0):
        q = torch.zeros(s.G, s.d)
        q[:, 0] = first
        q = q.to(T.DT[dtype])
        out = s.decode(q, None, None, None, [n - 1])
        s.check_out(out, q, [n - 1])
    assert int(s.err.item()) == 0


def turned(pos, turns):
    """(cos, sin) of 2 pi pos turns / 2^64 for int64 turns, in 64 bits: the angle's fraction from
    the integers."""
    frac = (np.asarray(pos, dtype=np.uint64)[..., None]
            * turns.cpu().numpy().astype(np.uint64)).astype(np.int64).astype(np.float64)
    angle = frac * (2 * np.pi / 2.0 ** 64)
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_rope_of_unit_pairs_is_cos_and_sin(d, half):
    """Pairs (1, 0) and (0, 1) give cos and sin themselves.  sincospif is off by one unit in the
    last place at most (2^-24 below 1), the first-order term's sum rounds by 2^-25, the fraction's
    bits past the 32nd are 2^-29.3 of an angle: 1.6 * 2^-24.  What a float's 24 bits lose of the
    angle, left out, would be up to pi 2^-25 = 1.57 * 2^-24 more."""
    n = 512
    p = fg.Params(1, 1, 2, n, d, fg.FG_FP32, 0.95, 0.3, 0.3, 0.0, 2)
    _, turns = T.table(d)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    first = slice(0, d // 2) if half else slice(0, d, 2)
    second = slice(d // 2, d) if half else slice(1, d, 2)
    x = torch.zeros(2, n, d)
    x[0, :, first] = 1.0
    x[1, :, second] = 1.0
    for start in (0, 100000, (1 << 30) + 7):
        pos = T.dev(torch.arange(start, start + n, dtype=torch.int32)[None])
        y = torch.empty(2, n, d, device="cuda")
        fg.fastgen_rope(p, None, T.dev(x), pos, rope, None, y)
        c, s = turned(np.arange(start, start + n), turns)
        y = T.f64(y)
        for got, want in ((y[0, :, first], c), (y[0, :, second], s),
                          (y[1, :, first], -s), (y[1, :, second], c)):
            assert np.abs(got - want).max() <= 1.6 * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,half", [(128, 128, False), (128, 64, True), (64, 32, False),
                                        (64, 64, True)])
def test_rope_is_near_its_definition(d, rot, half, dtype):
    """cos and sin within 1.6 * 2^-24, a product and a fused sum in 32 bits: 2^-22 of |x| + |y| of
    the pair, and the rounding to the type (bf16 2^-8)."""
    n, H = 300, 6
    p = fg.Params(2, 1, H, n, d, T.CODE[dtype], 0.95, 0.3, 0.3, 0.0, H)
    _, turns = T.table(rot)
    rope = fg.Rope(turns, fg.FG_ROPE_HALF if half else fg.FG_ROPE_INTERLEAVED)
    x = torch.randn(2 * H, n, d, generator=T.gen(d + rot)).to(T.DT[dtype])
    pos = torch.randint(0, 1 << 31, (2, n), generator=T.gen(1)).to(torch.int32)
    y = torch.empty_like(x, device="cuda")
    fg.fastgen_rope(p, T.dev(x), None, T.dev(pos), rope, y, None)
    c, s = (t.reshape(2, 1, n, rot // 2) for t in turned(pos.numpy(), turns))
    i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if half
            else (slice(0, rot, 2), slice(1, rot, 2)))
    x64, got = (T.f64(t).reshape(2, H, n, d) for t in (x, y))
    a, b = x64[..., i], x64[..., j]
    size = np.abs(a) + np.abs(b)
    for want, z in ((a * c - b * s, got[..., i]), (b * c + a * s, got[..., j])):
        bound = 2.0 ** -22 * size + (2.0 ** -8 if dtype == "bf16" else 0.0) * np.abs(want)
        assert (np.abs(z - want) <= bound).all()
    assert np.array_equal(got[..., rot:], x64[..., rot:])
