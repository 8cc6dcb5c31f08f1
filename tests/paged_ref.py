"""A plain float64 statement of the paged 8-bit caches, one cache at a time in
logical rows (no pages), and the reading of the GPU's pages into it.

A row's K (or V) values are codes * 2^e with one e per 16 rows: the least
e >= -100 with amax <= 448 * 2^e over the block's finite values, grown (and
the other codes rounded again) when a later row needs it.  e4m3: 4 significant
bits, exponents from -6, at most 448.
"""
import math

import numpy as np

PAGE, BLOCK, E_MIN, TOP = 64, 16, -100, 448.0
S, SP, SPF, SPFL, FULL = range(5)


def round_e4m3(x):
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), TOP)  # infinities too; NaN stays
    _, e = np.frexp(np.where(a > 0, a, 1.0))
    step = 2.0 ** (np.maximum(e - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, TOP), x)


def exponent(x):
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0)
    if top == 0.0:
        return E_MIN
    e = math.floor(math.log2(top)) - 12  # well below
    while top > TOP * 2.0 ** e:
        e += 1
    return max(e, E_MIN)


def rotate(x, pos, inv_freq, half):
    """x [..., d] at pos (broadcast against x without d), in float64."""
    y = np.array(x, dtype=np.float64)
    h = len(inv_freq)
    if h == 0:
        return y
    th = np.multiply.outer(np.asarray(pos, dtype=np.float64), inv_freq)
    c, s = np.cos(th), np.sin(th)
    i, j = (slice(0, h), slice(h, 2 * h)) if half else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


class Side:
    """K or V of one segment: codes [rows, d], block exponents."""

    def __init__(self, rows, d):
        self.codes = np.zeros((rows, d))
        self.e = np.full(-(-rows // BLOCK), E_MIN)

    def put(self, rows, values, fresh):
        """values of `rows` (distinct) in one go; fresh(block): it starts anew."""
        for b in sorted({r // BLOCK for r in rows}):
            mine = [i for i, r in enumerate(rows) if r // BLOCK == b]
            need = max(exponent(values[i]) for i in mine)
            sl = slice(b * BLOCK, (b + 1) * BLOCK)
            if not fresh(b):
                need = max(need, int(self.e[b]))
                if need > self.e[b]:
                    self.codes[sl] = round_e4m3(self.codes[sl] * 2.0 ** float(self.e[b] - need))
            self.e[b] = need
            for i in mine:
                self.codes[rows[i]] = round_e4m3(np.asarray(values[i]) * 2.0 ** float(-need))

    def values(self, rows):
        rows = np.asarray(rows, dtype=int)
        return self.codes[rows] * 2.0 ** self.e[rows // BLOCK][:, None].astype(float)


class RefCache:
    def __init__(self, policy, w, cap, d):
        self.policy, self.w, self.cap, self.d = policy, w if policy == SPFL else 0, cap, d
        self.rows = 0
        self.seg = {x: Side(cap, d) for x in "kv"}
        self.ring = {x: Side(-(-self.w // PAGE) * PAGE, d) for x in "kv"}
        self.seg_pos = np.full(cap, -1)
        self.ring_pos = np.full(self.w, -1)

    def compact(self, static, window, K, V):
        for x, X in (("k", K), ("v", V)):
            self.seg[x].put(list(range(len(static))), [X[j] for j in static], lambda b: True)
            self.ring[x].put([j % self.w for j in window], [X[j] for j in window], lambda b: True)
        self.rows = len(static)
        self.seg_pos[: self.rows] = static
        for j in window:
            self.ring_pos[j % self.w] = j

    def to_segment(self, special, punct):
        return self.policy == FULL or special or (self.policy != S and punct)

    def append(self, k, v, kinds, pos, room=None):
        """Rows k, v (rotated) of tokens at pos, pos + 1, ... with kinds (special, punct);
        room: rows the segment may reach."""
        m, old = len(k), self.rows
        room = self.cap if room is None else min(self.cap, room)
        st = [i for i in range(m) if self.to_segment(*kinds[i])][: max(room - old, 0)]
        ring = [i for i in range(max(m - self.w, 0), m)
                if self.w and not self.to_segment(*kinds[i])]
        slots = [(pos + i) % self.w for i in ring]
        for x, X in (("k", k), ("v", v)):
            self.seg[x].put(list(range(old, old + len(st))), [X[i] for i in st],
                            lambda b: b * BLOCK >= old)
            self.ring[x].put(slots, [X[i] for i in ring], lambda b: False)
        for r, i in enumerate(st):
            self.seg_pos[old + r] = pos + i
        for s, i in zip(slots, ring):
            self.ring_pos[s] = pos + i
        self.rows += len(st)

    def live(self, t):
        ring = [s for s in range(self.w) if self.ring_pos[s] >= 0 and t - self.w < self.ring_pos[s] <= t]
        return np.arange(self.rows), np.array(ring, dtype=int)

    def kv(self, t):
        """K, V of the live rows, and V's exponent of each."""
        a, b = self.live(t)
        k, v = (np.concatenate([self.seg[x].values(a), self.ring[x].values(b)]) for x in "kv")
        return k, v, np.concatenate([self.seg["v"].e[a // BLOCK], self.ring["v"].e[b // BLOCK]])


def attend(q, k, v, ev, scale):
    """(out, sum_j p_j |v_j|, max_j sum |q_i k_ji| times scale, floor) of one query: floor is
    2^-40 max_i(p_i 2^ev_i) sum_j |code_j|."""
    if len(k) == 0:
        z = np.zeros(q.shape[-1])
        return z, z, 0.0, z
    s = scale * (k @ q)
    p = np.exp(s - s.max())
    p /= p.sum()
    codes = np.abs(v) / 2.0 ** ev[:, None].astype(float)
    floor = 2.0 ** -40 * (p * 2.0 ** ev.astype(float)).max() * codes.sum(0)
    return p @ v, p @ np.abs(v), scale * float((np.abs(k) @ np.abs(q)).max()), floor


def decode_bound(out, weight, products, floor, dtype):
    """How far an output may be off.  The query carries 11 bits (fp16 rounding 2^-11 of each value)
    with bf16 inputs, 22 with fp32 (2^-22, plus what the second term loses); the sum over
    d <= 128 products in 32 bits adds at most 2^-20 of the sum of magnitudes (128 roundings of
    2^-24 and the tensor core's truncations); `products` bounds that sum times the scale.  A score
    off by ds changes each weight by a factor within e^(+-2 ds).  A weight is rounded once more,
    2^-11 (bf16) or 2^-21 (fp32), exponentials and sums in 32 bits add 2^-19; the result is
    rounded to its type (bf16 2^-8, fp32 2^-24).  floor: a weight w_j = p_j 2^ev_j enters as f16 of
    2^15 w_j / max w; where that is subnormal the steps are 2^-24, so it is off by at most
    2^-25 2^-15 max w, whatever its size, and so much times |code_j| is added for every row."""
    q = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
    ds = products * (q + 2.0 ** -20)
    rel = np.expm1(2 * ds) + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) * 2 + 2.0 ** -19
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    return rel * weight + floor * (1 + rel) + half * np.abs(out) + 1e-30


class GpuPages:
    """Host copies of a PagedCache's buffers, read by cache."""

    def __init__(self, cache):
        import torch

        n, d = cache.c.n_pages, cache.d
        self.codes = {x: getattr(cache, x + "_pages").reshape(n, PAGE, d).view(torch.float8_e4m3fn)
                      .float().cpu().numpy().astype(np.float64) for x in "kv"}
        self.e = cache.exps.reshape(n, PAGE // BLOCK, 2).cpu().numpy().astype(int)
        self.pos = cache.pos.reshape(n, PAGE).cpu().numpy().astype(int)
        self.table = cache.page_table.cpu().numpy().astype(int)
        self.caches = cache.caches.reshape(-1, 6).cpu().numpy().astype(int)
        self.rows = cache.rows_out.cpu().numpy().astype(int)

    def pages(self, c, ring):
        _, _, first, n, rfirst, rn = self.caches[c]
        return self.table[rfirst: rfirst + rn] if ring else self.table[first: first + n]

    def segment(self, c, ring, rows):
        """codes and exponents (K, V) and positions of the first `rows` rows."""
        pg = self.pages(c, ring)[: -(-rows // PAGE)]
        assert (pg >= 0).all(), (c, ring, pg)
        out = {}
        for which, x in enumerate("kv"):
            out[x] = self.codes[x][pg].reshape(-1, self.codes[x].shape[-1])[:rows]
            out["e" + x] = self.e[pg][:, :, which].reshape(-1)[: -(-rows // BLOCK)]
        out["pos"] = self.pos[pg].reshape(-1)[:rows]
        return out
