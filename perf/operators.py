"""Workloads of the paged 8-bit cache operators: what is timed and compared.

Four operators of the serving path of adaptive per-head caches:

  rope        rotation of a prompt's Q and K by position;
  compact_q8  the kept prompt rows of every cache, coded in 8 bits into pages;
  append_q8   new tokens' rows, rotated, placed by each cache's policy and
              coded into its pages;
  decode_q8   one generation step: the new token appended and every query head
              attending over its cache.

Data model (a cache belongs to one key/value head and serves its group's query
heads).  A page holds 64 rows of one cache: e4m3 codes [64, d] of K and of V,
the position of each row, and for every block of 16 rows one power-of-two
exponent of K and one of V: a row's value is code * 2^exponent.  The exponent
of a block is the least e with amax <= 448 * 2^e over the block's finite
values (not below -100).  When a later row needs a larger exponent, the codes
of the block are rounded again at the new one; a block whose first row is new
starts afresh.  A cache has a never-evicted segment of `rows` rows, and, for
the local hybrid, a ring of w rows in which position p lives at slot p mod w;
a ring row counts while its position is in (t - w, t].  page_table maps both
to pages.

With own = False the functions below compute that in elementary torch
operations; with own = True they make the framework's calls.
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK = 64, 16
E_MIN = -100
CODE_MAX = 448.0
SPECIAL = (1,)
PUNCT = (11, 402, 1753, 4810, 7777, 12011, 18943, 22222, 27001, 31999)
S, SP, SPF, SPFL, FULL = range(5)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _case(name, op, B, L, H, Hkv, n, d, dtype, gen=0, m=1, r_l=0.3, rot=0, style="interleaved",
          base=10000.0, start=0, idle=False):
    c = dict(op=op, B=B, L=L, H=H, Hkv=Hkv, n=n, d=d, dtype=dtype, gen=gen, m=m, r_l=r_l, rot=rot,
             style=style, base=base, start=start, idle=idle)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a chunk of a long prompt with grouped keys, half-rotated heads, far positions, odd length
        _case("rope-chunk-gqa", "rope", 2, 4, 32, 8, 1531, 128, "bf16", rot=64, style="half",
              base=500000.0, start=100000),
        # the 7B attention shape's prompt, eight layers of it
        _case("rope-7b", "rope", 1, 8, 32, 32, 2048, 128, "bf16", rot=128),
        # the 7B shape's prompt caches, eight layers
        _case("compact-7b", "compact", 1, 8, 32, 32, 2048, 128, "bf16"),
        # a long prompt, few heads
        _case("compact-32k", "compact", 1, 1, 8, 8, 32768, 128, "bf16", r_l=0.1),
        # fp32, small heads, grouped, odd length, two sequences
        _case("compact-odd-fp32", "compact", 2, 2, 16, 4, 777, 64, "fp32"),
        # the step's rows of every cache of the 7B shape (32 layers)
        _case("append-7b-one", "append", 1, 32, 32, 32, 2048, 128, "bf16", gen=37, m=1, rot=128),
        # accepted tokens of a speculative step, grouped keys, ragged batch with an idle sequence
        _case("append-gqa-few", "append", 8, 32, 32, 8, 1000, 128, "bf16", gen=11, m=5, rot=128,
              style="half", base=500000.0, idle=True),
        # a whole next turn, fp32, longer than the window
        _case("append-turn-fp32", "append", 2, 4, 16, 16, 900, 64, "fp32", gen=3, m=701, rot=64),
        # one layer's step on a short prompt: latency
        _case("decode-small", "decode", 1, 1, 32, 32, 128, 128, "bf16", gen=5, rot=128),
        # fp32, odd sizes, groups of two, no rotation
        _case("decode-odd-fp32", "decode", 3, 2, 8, 4, 501, 64, "fp32", gen=9),
        # the 7B shape, every layer
        _case("decode-7b", "decode", 1, 32, 32, 32, 2048, 128, "bf16", gen=100, rot=128),
        # grouped keys, long prompt, a batch with an idle sequence
        _case("decode-gqa-16k", "decode", 4, 8, 64, 8, 16384, 128, "bf16", gen=64, rot=128,
              r_l=0.1, style="half", base=500000.0, idle=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("rope", "compact", "append", "decode"))
        d, dtype = rng.choice((64, 128)), rng.choice(("bf16", "bf16", "fp32"))
        B, L = _log(rng, 1, 8), _log(rng, 1, 16)
        Hkv = rng.choice((1, 2, 4, 8, 8, 32))
        H = Hkv * rng.choice((1, 1, 2, 4, 8))
        n = _log(rng, 1, 20000)
        rot = rng.choice((0, d // 2, d)) if op != "rope" else rng.choice((d // 2, d))
        c = _case(None, op, B, L, H, Hkv, n, d, dtype, gen=_log(rng, 1, 200),
                  m=_log(rng, 1, 800) if op == "append" else 1,
                  r_l=round(rng.uniform(0.0, 0.4), 3), rot=rot,
                  style=rng.choice(("interleaved", "half")),
                  base=rng.choice((10000.0, 500000.0)), start=_log(rng, 1, 1 << 20) - 1,
                  idle=B >= 2 and rng.random() < 0.3)
        if _gkv(c) * n * d <= 1.2e8 and _gkv(c) <= 1024 and work(c)["bytes"] <= 5e8 \
                and _gkv(c) * c["m"] * d <= 3e7 and _rows(c).sum() >= 1:
            return c


# ------------------------------------------- what is the same for every seed
def _gkv(c):
    return c["B"] * c["L"] * c["Hkv"]


def _window(c):
    return int(math.ceil(float(np.float32(c["r_l"])) * c["n"]))


def _policies(c):
    """Shortlist entry of each cache: 15 % special, 20 % punct, 10 % frequent, 25 % local, 30 % full."""
    kind = (np.arange(_gkv(c)) * 13 + 5) % 20
    return np.select([kind < 3, kind < 7, kind < 9, kind < 14], [S, SP, SPF, SPFL], FULL)


def _kept(c):
    """Never-evicted prompt rows of each cache (some special-only caches are empty)."""
    pol, n, i = _policies(c), c["n"], np.arange(_gkv(c))
    want = np.select([pol == S, pol == SP, pol == SPF, pol == SPFL],
                     [i % 3, 1 + n // 20 + i % 7, 1 + (3 * n) // 10 + i % 17,
                      1 + (8 * n) // 25 + i % 17], n)
    return np.minimum(want, n).astype(np.int64)


def _rows(c):
    """Never-evicted rows of each cache when the timed call begins."""
    pol, gen = _policies(c), c["gen"] if c["op"] in ("append", "decode") else 0
    grown = np.select([pol == S, pol == FULL], [0, gen], gen // 20)
    return _kept(c) + grown


def _ring(c):
    return np.where(_policies(c) == SPFL, _window(c), 0).astype(np.int64)


def _seq(c):
    return np.arange(_gkv(c)) // (c["L"] * c["Hkv"])


def _live(c):
    """Sequences that take part (an idle one has position -1)."""
    b = np.arange(c["B"])
    return b != c["B"] - 1 if c["idle"] and c["op"] in ("append", "decode") else b >= 0


def _new_counts(c):
    """New tokens of each sequence: ragged when several are appended."""
    b = np.arange(c["B"])
    return np.where(_live(c), np.maximum(c["m"] - b % 3, 1), 0).astype(np.int64)


# ------------------------------------------------------------------ inputs
def _inv_freq(c):
    return c["base"] ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / max(c["rot"], 1))


def _layout(c, rows, grow):
    """caches [Gkv, 6] (policy, w, first table entry and entries of the never-evicted segment,
    first table entry and entries of the ring) and the number of table entries."""
    seg = np.maximum(1, -(-(rows + grow) // PAGE))
    w = _ring(c)
    ring = -(-w // PAGE)
    first = np.concatenate([[0], np.cumsum(seg + ring)[:-1]])
    return np.stack([_policies(c), w, first, seg, first + seg, ring], 1).astype(np.int32), \
        int((seg + ring).sum())


def _values(g, shape, dtype, channels):
    """Normal values with the spread of real keys: per-cache sizes and, for keys, a few large
    channels."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g,
                                     device="cuda"))
    if channels:
        x[..., 3::29] *= 4.0
    return x.to(dtype)


def _token_ids(g, shape):
    ids = torch.randint(2, 32000, shape, generator=g, device="cuda", dtype=torch.int32)
    pick = torch.rand(shape, generator=g, device="cuda")
    punct = torch.tensor(PUNCT, dtype=torch.int32, device="cuda")
    ids = torch.where(pick < 0.05, punct[(ids % len(PUNCT)).long()], ids)
    return torch.where(pick > 0.99, torch.full_like(ids, SPECIAL[0]), ids)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt, G, gk, n, d = DTYPES[c["dtype"]], c["B"] * c["L"] * c["H"], _gkv(c), c["n"], c["d"]
    s = dict(case=c, special=torch.tensor(SPECIAL, dtype=torch.int32, device=dev),
             punct=torch.tensor(PUNCT, dtype=torch.int32, device=dev),
             dev_err=torch.zeros(1, dtype=torch.int32, device=dev))
    inv = _inv_freq(c)
    s["inv_freq"] = torch.from_numpy(inv).to(dev)
    # turns a position, as 64-bit fractions: what the framework's rotation takes
    s["turns"] = torch.tensor([int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in inv],
                              dtype=torch.int64, device=dev)
    if c["op"] == "rope":
        s["Q"] = _values(g, (G, n, d), dt, False)
        s["K"] = _values(g, (gk, n, d), dt, True)
        first = c["start"] + 17 * torch.arange(c["B"], device=dev, dtype=torch.int32)
        s["pos"] = (first[:, None] + torch.arange(n, device=dev, dtype=torch.int32)[None]
                    ).contiguous()
        s["Q_out"], s["K_out"] = torch.zeros_like(s["Q"]), torch.zeros_like(s["K"])
    else:
        rows, w = _rows(c), _window(c)
        caches, entries = _layout(c, rows, 0 if c["op"] == "compact" else c["m"] + 8)
        s["caches"] = torch.from_numpy(caches).to(dev)
        # pages in no particular order, as in a pool that other sequences have used
        s["page_table"] = torch.randperm(entries, generator=g, device=dev).to(torch.int32)
        s["rows"] = torch.from_numpy(rows.astype(np.int32)).to(dev)
        s["rows_out"] = s["rows"].clone()
        s["next_page"] = torch.tensor([entries], dtype=torch.int32, device=dev)
        s["most"] = (int(caches[:, 3].max()), int(caches[:, 5].max()))
        s["k"] = torch.zeros((entries, PAGE, d), dtype=torch.float8_e4m3fn, device=dev)
        s["v"] = torch.zeros_like(s["k"])
        s["exps"] = torch.full((entries, PAGE // BLOCK, 2), E_MIN, dtype=torch.int8, device=dev)
        s["pos_pages"] = torch.full((entries, PAGE), -1, dtype=torch.int32, device=dev)
        if c["op"] == "compact":
            s["K"], s["V"] = _values(g, (gk, n, d), dt, True), _values(g, (gk, n, d), dt, False)
            s["keep"] = _keep(c, g)
        else:
            live = torch.from_numpy(_live(c)).to(dev)
            at = n + c["gen"] + 3 * torch.arange(c["B"], device=dev, dtype=torch.int32)
            s["pos"] = torch.where(live, at, torch.full_like(at, -1))
            s["n_new"] = torch.from_numpy(_new_counts(c).astype(np.int32)).to(dev)
            _fill(s, g)
            m = c["m"]
            many = (m,) if c["op"] == "append" else ()
            s["ids"] = _token_ids(g, (c["B"],) + many)
            s["k_new"] = _values(g, (gk,) + many + (d,), dt, True)
            s["v_new"] = _values(g, (gk,) + many + (d,), dt, False)
            if c["op"] == "decode":
                s["q"] = _values(g, (G, d), dt, False)
                s["out"] = torch.zeros((G, d), dtype=dt, device=dev)
    if own:
        _handles(s)
    return s


def _keep(c, g):
    """Keep codes [G, n]: member 0 of a group holds its cache's set, the others part of it."""
    gk, n, R = _gkv(c), c["n"], c["H"] // c["Hkv"]
    kept = torch.from_numpy(_kept(c)).cuda()
    order = torch.rand((gk, n), generator=g, device="cuda").argsort(1).argsort(1)
    st = order < kept[:, None]
    w = torch.from_numpy(_ring(c)).cuda()
    win = torch.arange(n, device="cuda")[None] >= n - w[:, None]
    code = torch.where(st, 1, torch.where(win, 2, 0)).to(torch.uint8)
    part = torch.rand((gk, R, n), generator=g, device="cuda") < 0.5
    part[:, 0] = True
    return torch.where(part, code[:, None], torch.zeros_like(code)[:, None]).reshape(-1, n)


def _fill(s, g):
    """A cache in use: rows of the prompt and of earlier steps, coded."""
    c = s["case"]
    e, d = s["k"].shape[0], c["d"]
    step = 4096
    for a in range(0, e, step):
        z = min(e, a + step)
        for key, channels, which in (("k", True, 0), ("v", False, 1)):
            x = _values(g, (z - a, PAGE, d), torch.float32, channels).view(-1, BLOCK, d)
            ex = _exponent(x.abs().amax((1, 2)))
            s[key][a:z] = _code(x, ex[:, None, None]).view(z - a, PAGE, d)
            s["exps"][a:z, :, which] = ex.view(z - a, -1).to(torch.int8)
    # the ring's positions: a slot whose token went to the never-evicted segment keeps an older one
    seq = torch.from_numpy(_seq(c)).cuda()
    t = s["pos"].long()[seq].clamp(min=0) - 1
    w = s["caches"][:, 1].long()
    tables, pages = _pages(s, 4, s["most"][1])
    slot = torch.arange(s["most"][1] * PAGE, device="cuda")[None]
    p = t[:, None] - (t[:, None] - slot) % w.clamp(min=1)[:, None]
    old = torch.rand(p.shape, generator=g, device="cuda") < 0.06
    p = torch.where(old, p - w[:, None], p)
    ok = (slot < w[:, None]) & tables.repeat_interleave(PAGE, 1)
    at = pages.repeat_interleave(PAGE, 1) * PAGE + slot % PAGE
    s["pos_pages"].view(-1)[at[ok]] = p[ok].clamp(min=-1).to(torch.int32)


def _pages(s, first, most):
    """(is there such a page, its number) for the first `most` pages of a segment of each cache:
    column `first` of caches holds its first table entry, the next column (or the one of the
    never-evicted segment) its entries."""
    cc = s["caches"].long()
    j = torch.arange(most, device="cuda")[None]
    ok = j < cc[:, first + 1, None]
    at = torch.where(ok, cc[:, first, None] + j, 0)
    return ok, s["page_table"].long()[at]


# ------------------------------------------------------------ the framework
def _handles(s):
    from adaptive_head_kv_gb300 import fastgen as fg

    c = s["case"]
    code = {"bf16": fg.FG_BF16, "fp32": fg.FG_FP32}[c["dtype"]]
    s["p"] = fg.Params(c["B"], c["L"], c["H"], c["n"], c["d"], code, 0.95, c["r_l"], 0.3, 0.0,
                       c["Hkv"])
    s["rope"] = None
    if c["rot"]:
        s["rope"] = fg.Rope(s["turns"], style={"interleaved": fg.FG_ROPE_INTERLEAVED,
                                               "half": fg.FG_ROPE_HALF}[c["style"]])
    if c["op"] == "rope":
        return
    s["cache"] = fg.PagedCache(s["p"], s["k"], s["v"], s["exps"], s["pos_pages"],
                               s["page_table"], s["caches"], s["rows"], s["next_page"],
                               rows_out=s["rows_out"])
    if c["op"] == "append":
        need = fg.fastgen_append_q8_workspace_bytes(s["p"], c["m"])
        s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    if c["op"] == "decode":
        s["cache"].schedule(s["p"])
        need = fg.fastgen_decode_q8_workspace_bytes(s["p"], s["cache"])
        s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")


def _run_own(s):
    from adaptive_head_kv_gb300 import fastgen as fg

    op = s["case"]["op"]
    if op == "rope":
        fg.fastgen_rope(s["p"], s["Q"], s["K"], s["pos"], s["rope"], s["Q_out"], s["K_out"])
    elif op == "compact":
        fg.fastgen_compact_q8(s["p"], s["K"], s["V"], s["keep"], s["cache"], s["dev_err"])
    elif op == "append":
        fg.fastgen_append_q8(s["p"], s["cache"], s["k_new"], s["v_new"], s["ids"], s["n_new"],
                             s["special"], s["punct"], s["pos"], s["rope"], s["ws"],
                             s["dev_err"])
    else:
        fg.fastgen_decode_attn_q8(s["p"], s["cache"], s["q"], s["k_new"], s["v_new"], s["ids"],
                                  s["special"], s["punct"], s["pos"], s["rope"], s["out"],
                                  s["ws"], s["dev_err"])


def _outputs(s):
    op = s["case"]["op"]
    if op == "rope":
        return dict(q=s["Q_out"], k=s["K_out"])
    o = dict(k=s["k"], v=s["v"], exps=s["exps"], pos=s["pos_pages"])
    if op != "compact":
        o["rows"] = s["rows_out"]
    if op == "decode":
        o["out"] = s["out"]
    return o


def run(state):
    if own:
        _run_own(state)
    else:
        dict(rope=_rope_plain, compact=_compact_plain, append=_append_plain,
             decode=_decode_plain)[state["case"]["op"]](state)
    return _outputs(state)


# ------------------------------------------------------------- plain forms
def _exponent(amax):
    """Least e >= E_MIN with amax <= 448 * 2^e, from the number's own exponent and fraction."""
    bits = amax.float().view(torch.int32)
    e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(min=E_MIN)


def _pow2(e):
    return torch.exp2(e.double())


def _code(x, e):
    """e4m3 codes of x * 2^-e, nearest even; infinities become the largest code."""
    y = (x.double() * _pow2(-e)).float().clamp(-CODE_MAX, CODE_MAX)
    return y.to(torch.float8_e4m3fn)


def _amax(x, dim):
    a = x.float().abs()
    return torch.where(torch.isfinite(a), a, torch.zeros_like(a)).amax(dim)


def _rotated(x, pos, c, inv_freq):
    """x [..., d] in 32 bits, rotated at pos (the shape of x without d, or broadcastable to it)."""
    x, rot = x.float(), c["rot"]
    if not rot:
        return x
    angle = pos.double()[..., None] * inv_freq
    cos, sin = angle.cos().float(), angle.sin().float()
    if c["style"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _rope_plain(s):
    c = s["case"]
    for key in ("Q", "K"):
        x = s[key].view(c["B"], -1, c["n"], c["d"])
        y = _rotated(x, s["pos"][:, None], c, s["inv_freq"])
        s[key + "_out"].copy_(y.view(s[key].shape))


def _write_rows(s, at, xk, xv, fresh):
    """Codes rows xk, xv [r, d] into pool rows `at` [r]; fresh [r]: the row's block starts anew.
    Other rows of a block whose exponent grows are rounded again."""
    blocks = at // BLOCK
    nb, d = s["k"].shape[0] * (PAGE // BLOCK), s["case"]["d"]
    touched = torch.zeros(nb, dtype=torch.bool, device="cuda")
    touched[blocks] = True
    anew = torch.zeros(nb, dtype=torch.bool, device="cuda")
    anew[blocks] = fresh
    ids = touched.nonzero()[:, 0]
    for key, x, which in (("k", xk, 0), ("v", xv, 1)):
        need = torch.full((nb,), -128, dtype=torch.int32, device="cuda")
        need.scatter_reduce_(0, blocks, _exponent(_amax(x, -1)), "amax")
        had = s["exps"].view(nb, 2)[:, which].int()
        had = torch.where(anew, torch.full_like(had, -128), had)
        now = torch.maximum(need, had)
        codes = s[key].view(torch.uint8).view(nb, BLOCK, d)
        shift = torch.where(anew, torch.zeros_like(now), had - now)[ids]
        old = codes[ids].view(torch.float8_e4m3fn).float()
        codes[ids] = (old * _pow2(shift).float()[:, None, None]).to(torch.float8_e4m3fn).view(
            torch.uint8)
        s[key].view(torch.uint8).view(-1, d)[at] = _code(x, now[blocks][:, None]).view(torch.uint8)
        s["exps"].view(nb, 2)[:, which][ids] = now[ids].to(torch.int8)


def _compact_plain(s):
    c = s["case"]
    gk, n, d, R, hkv = _gkv(c), c["n"], c["d"], c["H"] // c["Hkv"], c["Hkv"]
    keep = s["keep"].view(-1, hkv, R, n)
    st = (keep == 1).any(2).view(gk, n)
    win = (keep == 2).any(2).view(gk, n) & ~st
    cc, table = s["caches"].long(), s["page_table"].long()
    j = torch.arange(n, device="cuda")[None]
    row = torch.where(st, st.cumsum(1) - 1, j % cc[:, 1, None].clamp(min=1))
    entry = torch.where(st, cc[:, 2, None], cc[:, 4, None]) + row // PAGE
    kept = st | win
    at = (table[torch.where(kept, entry, 0)] * PAGE + row % PAGE)[kept]
    # ring slots first empty, their blocks (and the segment's) at the least exponent
    ok, pages = _pages(s, 4, s["most"][1])
    slot = torch.arange(s["most"][1] * PAGE, device="cuda")[None]
    live = ok.repeat_interleave(PAGE, 1) & (slot < cc[:, 1, None])
    ring = (pages.repeat_interleave(PAGE, 1) * PAGE + slot % PAGE)[live]
    s["pos_pages"].view(-1)[ring] = -1
    s["exps"].view(-1, 2)[ring // BLOCK] = E_MIN
    s["exps"].view(-1, 2)[at // BLOCK] = E_MIN
    s["pos_pages"].view(-1)[at] = j.expand(gk, n)[kept].to(torch.int32)
    _write_rows(s, at, s["K"][kept], s["V"][kept], torch.ones_like(at, dtype=torch.bool))


def _append_plain(s):
    c = s["case"]
    gk, d = _gkv(c), c["d"]
    m = c["m"] if c["op"] == "append" else 1
    seq = torch.arange(gk, device="cuda") // (c["L"] * c["Hkv"])
    cc, table = s["caches"].long(), s["page_table"].long()
    ids = s["ids"].view(c["B"], m)
    special = (ids[..., None] == s["special"]).any(-1)
    punct = (ids[..., None] == s["punct"]).any(-1)
    pol, w, rows = cc[:, 0, None], cc[:, 1, None], s["rows"].long()[:, None]
    to_static = (pol == FULL) | special[seq] | ((pol != S) & punct[seq])
    i = torch.arange(m, device="cuda")[None]
    pos = s["pos"].long()[seq][:, None]
    count = s["n_new"].long()[seq][:, None] if c["op"] == "append" else 1
    active = (pos >= 0) & (i < count)
    st = to_static & active
    row = rows + st.cumsum(1) - 1
    st = st & (row < cc[:, 3, None] * PAGE)
    ring = ~to_static & active & (pol == SPFL) & (w > 0) & (i >= count - w)
    slot = (pos + i) % w.clamp(min=1)
    place = torch.where(st, row, slot)
    entry = torch.where(st, cc[:, 2, None], cc[:, 4, None]) + place // PAGE
    put = st | ring
    at = table[torch.where(put, entry, 0)] * PAGE + place % PAGE
    fresh = st & (row - row % BLOCK >= rows)
    k = _rotated(s["k_new"].view(gk, m, d), pos + i, c, s["inv_freq"])
    v = s["v_new"].view(gk, m, d).float()
    _write_rows(s, at[put], k[put], v[put], fresh[put])
    s["pos_pages"].view(-1)[at[put]] = (pos + i).expand(gk, m)[put].to(torch.int32)
    s["rows_out"].copy_((rows[:, 0] + st.sum(1)).to(torch.int32))


def _decode_plain(s):
    _append_plain(s)
    c = s["case"]
    gk, d, R = _gkv(c), c["d"], c["H"] // c["Hkv"]
    seq = torch.arange(gk, device="cuda") // (c["L"] * c["Hkv"])
    cc = s["caches"].long()
    a, pa = _pages(s, 2, s["most"][0])
    b, pb = _pages(s, 4, s["most"][1])
    pages = torch.cat([pa, pb], 1)
    row = torch.arange(pa.shape[1] * PAGE, device="cuda")[None]
    slot = torch.arange(pb.shape[1] * PAGE, device="cuda")[None]
    t = s["pos"].long()[seq][:, None]
    p = s["pos_pages"][pb].view(gk, -1)
    w = cc[:, 1, None]
    ok = torch.cat([a.repeat_interleave(PAGE, 1) & (row < s["rows_out"].long()[:, None]),
                    b.repeat_interleave(PAGE, 1) & (slot < w) & (p >= 0) & (p > t - w) & (p <= t)],
                   1)
    q = _rotated(s["q"].view(c["B"], -1, d), s["pos"].clamp(min=0)[:, None], c, s["inv_freq"])
    q = q.view(gk, R, d) / math.sqrt(d)
    scale = _pow2(s["exps"][pages].int()).float().repeat_interleave(BLOCK, 2)

    def rows_of(key, which):
        x = s[key].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        return (x * scale[..., which, None]).view(gk, -1, d)

    score = torch.matmul(q, rows_of("k", 0).transpose(1, 2))
    score = score.masked_fill(~ok[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e / total.clamp(min=1e-30), rows_of("v", 1).masked_fill(~ok[..., None], 0.0))
    active = (t >= 0)[..., None]
    s["out"].copy_(torch.where(active, o, s["out"].view(gk, R, d).float()).view(-1, d))


# ----------------------------------------------------------------- the work
def work(case):
    c = case
    eb = 2 if c["dtype"] == "bf16" else 4
    G, gk, n, d, R = c["B"] * c["L"] * c["H"], _gkv(c), c["n"], c["d"], c["H"] // c["Hkv"]
    if c["op"] == "rope":
        return dict(bytes=2 * eb * (G + gk) * n * d + 4 * c["B"] * n,
                    flops=3 * (G + gk) * n * c["rot"])
    w, rows = _ring(c), _rows(c)
    if c["op"] == "compact":
        kept = rows + np.minimum(w, n - rows) * 0.68  # window rows that are not never-evicted ones
        k = float(kept.sum())
        return dict(bytes=k * (2 * eb * d + 2 * d + 4) + G * n + k / 8, flops=6 * k * d)
    live = _live(c)[_seq(c)]
    if c["op"] == "append":
        pol, new = _policies(c), np.where(live, _new_counts(c)[_seq(c)], 0)
        put = np.select([pol == S, (pol == SP) | (pol == SPF), pol == SPFL],
                        [0.01 * new, 0.06 * new, 0.06 * new + 0.94 * np.minimum(new, w)], new)
        k = float(put.sum())
        return dict(bytes=k * (2 * eb * d + 2 * d + 4) + 4 * c["B"] * c["m"] + 8 * gk,
                    flops=k * (6 * d + 3 * c["rot"]))
    att = float(((rows + w) * live).sum())
    nl = float(live.sum())
    return dict(bytes=att * 2 * d + att / 8 + 4 * float((w * live).sum()) + nl * (2 * R + 4) * eb * d,
                flops=4 * R * att * d + 3 * nl * (R + 1) * c["rot"])


# ---------------------------------------------------- the definition, 64 bits
def _round_code(y):
    """Nearest e4m3 value of y (numpy, 64 bits): three fraction bits, exponents from -6."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), CODE_MAX)
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, CODE_MAX), y)


def _least_exponent(amax):
    if not amax > 0:
        return E_MIN
    f, e = math.frexp(float(amax) / CODE_MAX)
    return max(E_MIN, e - 1 if f == 0.5 else e)


def _turn(x, p, c):
    """One row (or rows, with p of their number) rotated in 64 bits."""
    x = np.array(x, dtype=np.float64)
    rot = c["rot"]
    th = np.asarray(p, dtype=np.float64)[..., None] * _inv_freq(c)
    z = np.exp(1j * th)
    if rot and c["style"] == "half":
        u = (x[..., : rot // 2] + 1j * x[..., rot // 2: rot]) * z
        x[..., : rot // 2], x[..., rot // 2: rot] = u.real, u.imag
    elif rot:
        u = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * z
        x[..., 0:rot:2], x[..., 1:rot:2] = u.real, u.imag
    return x


def exact(case, seed):
    c = case
    w = work(c)
    if w["bytes"] > 6e8 and c["op"] != "decode":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "rope":
        return {key.lower(): torch.from_numpy(_turn(
            s[key].double().cpu().numpy().reshape(c["B"], -1, c["n"], c["d"]),
            s["pos"].cpu().numpy()[:, None], c)).view(s[key].shape) for key in ("Q", "K")}
    st = _Pages(s)
    (st.compact if c["op"] == "compact" else st.append)()
    o = dict(k=torch.from_numpy(st.k), v=torch.from_numpy(st.v), exps=None, pos=None)
    if c["op"] != "compact":
        o["rows"] = None
    if c["op"] == "decode":
        o["out"] = st.attend()
    return o


class _Pages:
    """The caches on the host, in 64 bits, changed a block at a time."""

    def __init__(self, s):
        self.s, self.c = s, s["case"]
        self.k, self.v = (s[x].double().cpu().numpy() for x in "kv")
        self.e = s["exps"].cpu().numpy().astype(np.int64)
        self.p = s["pos_pages"].cpu().numpy().astype(np.int64)
        self.caches = s["caches"].cpu().numpy().astype(np.int64)
        self.table = s["page_table"].cpu().numpy().astype(np.int64)
        self.rows = s["rows"].cpu().numpy().astype(np.int64)

    def block(self, first, b):
        page = self.table[first + b * BLOCK // PAGE]
        r = b * BLOCK % PAGE
        return page, r, r // BLOCK

    def put(self, first, b, fresh, lines):
        """lines: {row of the block: (key row, value row, position)}."""
        page, r, sub = self.block(first, b)
        for which, pool in ((0, self.k), (1, self.v)):
            x = {i: y[which] for i, y in lines.items()}
            now = max(_least_exponent(np.abs(y)[np.isfinite(y)].max(initial=0.0))
                      for y in x.values())
            if not fresh:
                now = max(now, self.e[page, sub, which])
                if now > self.e[page, sub, which]:
                    pool[page, r: r + BLOCK] = _round_code(
                        pool[page, r: r + BLOCK] * 2.0 ** (self.e[page, sub, which] - now))
            for i, y in x.items():
                pool[page, r + i] = _round_code(y * 2.0 ** -float(now))
            self.e[page, sub, which] = now
        for i, y in lines.items():
            self.p[page, r + i] = y[2]

    def compact(self):
        c, s = self.c, self.s
        R = c["H"] // c["Hkv"]
        keep = s["keep"].cpu().numpy()
        K, V = (s[x].double().cpu().numpy() for x in "KV")
        for g, (pol, w, first, _, ring, _) in enumerate(self.caches):
            codes = keep[g * R: (g + 1) * R]
            fixed = (codes == 1).any(0)
            static = np.flatnonzero(fixed)
            window = np.flatnonzero((codes == 2).any(0) & ~fixed)
            blocks = {}
            for r, j in enumerate(static):
                blocks.setdefault((first, r // BLOCK), {})[r % BLOCK] = (K[g, j], V[g, j], j)
            for j in window:
                blocks.setdefault((ring, j % w // BLOCK), {})[j % w % BLOCK] = (K[g, j], V[g, j], j)
            for (at, b), lines in blocks.items():
                self.put(at, b, True, lines)

    def append(self):
        c, s = self.c, self.s
        one = c["op"] == "decode"
        m = 1 if one else c["m"]
        gk, d = len(self.caches), c["d"]
        ids = s["ids"].cpu().numpy().reshape(-1, m)
        pos = s["pos"].cpu().numpy().astype(np.int64)
        count = np.ones(c["B"], np.int64) if one else s["n_new"].cpu().numpy()
        k, v = (s[x].double().cpu().numpy().reshape(gk, m, d) for x in ("k_new", "v_new"))
        for g, (pol, w, first, cap, ring, _) in enumerate(self.caches):
            b = g // (c["L"] * c["Hkv"])
            if pos[b] < 0:
                continue
            blocks, old = {}, self.rows[g]
            for i in range(count[b]):
                tok, t = int(ids[b, i]), int(pos[b]) + i
                if pol == FULL or tok in SPECIAL or (pol != S and tok in PUNCT):
                    r = self.rows[g]
                    if r >= cap * PAGE:
                        continue
                    self.rows[g] += 1
                    key = (first, r // BLOCK, r - r % BLOCK >= old)
                elif pol == SPFL and w > 0 and i >= count[b] - w:
                    r = t % w
                    key = (ring, r // BLOCK, False)
                else:
                    continue
                blocks.setdefault(key, {})[r % BLOCK] = (_turn(k[g, i], t, c), v[g, i], t)
            for (at, blk, fresh), lines in blocks.items():
                self.put(at, blk, fresh, lines)

    def attend(self):
        c, s = self.c, self.s
        R, d = c["H"] // c["Hkv"], c["d"]
        pos = s["pos"].cpu().numpy().astype(np.int64)
        q = s["q"].double().cpu().numpy()
        out = torch.zeros(q.shape, dtype=torch.float64)
        kd, vd = torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda()
        e = torch.exp2(torch.from_numpy(self.e).cuda().double())
        for g, (pol, w, first, cap, ring, _) in enumerate(self.caches):
            b = g // (c["L"] * c["Hkv"])
            if pos[b] < 0:
                continue
            r = np.arange(self.rows[g])
            at = [self.table[first + r // PAGE] * PAGE + r % PAGE]
            if w > 0:
                r = np.arange(w)
                z = self.table[ring + r // PAGE] * PAGE + r % PAGE
                p = self.p.reshape(-1)[z]
                at.append(z[(p >= 0) & (p > pos[b] - w) & (p <= pos[b])])
            at = np.concatenate(at)
            if not len(at):
                continue
            z = torch.from_numpy(at).cuda()
            sc = e.view(-1, 2)[z // BLOCK]
            kk, vv = (x.view(-1, d)[z] * sc[:, i, None] for i, x in ((0, kd), (1, vd)))
            qq = torch.from_numpy(_turn(q[g * R: (g + 1) * R], np.full(R, pos[b]), c)).cuda()
            out[g * R: (g + 1) * R] = (torch.softmax(qq @ kk.T / math.sqrt(d), -1) @ vv).cpu()
        return out
