"""Workloads of the serving operators beside plain paged decoding: what is timed and compared.

Three operators on paged 8-bit caches of a batch of sequences:

  shared  one generation step of sequences that continue one prompt: every
          query attends over the prompt's caches, which are there once, and
          over its own sequence's cache of what came since;
  weigh   one generation step that also adds to every never-evicted row the
          attention weight the step gives it (of all query heads of its group);
  evict   caches that have outgrown a budget of rows are cut to it: the newest
          rows stay, and of the others those of most accumulated weight.

Data model (a cache belongs to one key/value head and serves its group's query
heads).  A page holds 64 rows of one cache: e4m3 codes [64, d] of K and of V,
the position of each row, and for every block of 16 rows one power-of-two
exponent of K and one of V: a row's value is code * 2^exponent.  The exponent
of a block is the least e with amax <= 448 * 2^e over the block's finite
values (not below -100); when a later row needs a larger one, the block's codes
are rounded again at it; a block whose first row is new starts afresh.  A cache
has a never-evicted segment of `rows` rows, and, for the local hybrid, a ring
of w rows in which position p lives at slot p mod w; a ring row counts while
its position is in (t - w, t].  page_table maps both to pages.  scores
[pages, 64] holds the accumulated weight of the never-evicted rows, +inf for
rows that are never dropped.

Eviction keeps exactly `budget` rows of a longer segment: first the rows of
positions (t - recent, t], then by larger score (NaN and negative ones as 0),
ties to the lower row.  Kept rows below `budget` stay where they are; the
others move, in order, into the places of the dropped rows below it, and are
coded again at the exponents of the blocks they come to.

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
def _case(name, op, B, L, H, Hkv, n, d, dtype="bf16", gen=0, r_l=0.3, rot=0, style="interleaved",
          base=10000.0, idle=False, scores=False, budget=0, recent=0):
    c = dict(op=op, B=B, L=L, H=H, Hkv=Hkv, n=n, d=d, dtype=dtype, gen=gen, r_l=r_l, rot=rot,
             style=style, base=base, idle=idle, scores=scores or op == "weigh", budget=budget,
             recent=recent)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # four samples of one prompt, one layer: latency
        _case("shared-small", "shared", 4, 1, 32, 32, 1000, 128, gen=5, rot=128),
        # a batch behind one long system prompt, grouped keys, one layer
        _case("shared-gqa-8k", "shared", 16, 1, 32, 8, 8192, 128, gen=64, r_l=0.1, rot=128,
              style="half", base=500000.0),
        # a large batch of groups of 8 behind a long document, four layers
        _case("shared-gqa-16k", "shared", 64, 4, 64, 8, 16384, 128, gen=100, r_l=0.05, rot=128,
              style="half", base=500000.0),
        # many samples of one prompt, eight layers of the 7B attention shape
        _case("shared-7b", "shared", 64, 8, 32, 32, 4096, 128, gen=40, r_l=0.1, rot=128),
        # fp32, groups of 2, odd sizes, an idle sequence, half of the row rotated; weights are kept
        _case("shared-odd-fp32", "shared", 5, 2, 12, 6, 777, 64, "fp32", gen=70, rot=32, idle=True,
              scores=True),
        # fp32, groups of 4
        _case("shared-fp32", "shared", 24, 2, 32, 8, 4096, 128, "fp32", gen=33, r_l=0.1, rot=128),
        # fp32, odd sizes, groups of 2, no rotation
        _case("weigh-odd-fp32", "weigh", 3, 2, 8, 4, 501, 64, "fp32", gen=9),
        # the 7B shape, every layer
        _case("weigh-7b", "weigh", 1, 32, 32, 32, 2048, 128, gen=100, rot=128),
        # groups of 8, a longer prompt, an idle sequence
        _case("weigh-gqa-8k", "weigh", 4, 8, 64, 8, 8192, 128, gen=64, rot=128, r_l=0.1,
              style="half", base=500000.0, idle=True),
        # a ragged batch of small caches, some within their budget, an idle sequence
        _case("evict-odd", "evict", 3, 3, 8, 8, 500, 64, gen=130, budget=304, recent=37, idle=True),
        # the 7B shape, a quarter over its budget
        _case("evict-7b", "evict", 1, 32, 32, 32, 1024, 128, gen=256, budget=1024, recent=128),
        # the first cut of a long prompt's caches
        _case("evict-32k", "evict", 1, 2, 32, 8, 32768, 128, gen=1, budget=8192, recent=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(("shared", "shared", "weigh", "evict"))
        d, dtype = rng.choice((64, 128, 128)), rng.choice(("bf16", "bf16", "fp32"))
        B, L = _log(rng, 1, 96 if op == "shared" else 8), _log(rng, 1, 12)
        Hkv = rng.choice((1, 2, 4, 8, 8, 32))
        H = Hkv * rng.choice((1, 1, 2, 4, 8))
        n = _log(rng, 1, 20000)
        budget = recent = 0
        if op == "evict":
            dtype, budget = "bf16", BLOCK * _log(rng, 1, max(1, n // BLOCK))
            recent = rng.randrange(0, budget + 1)
        c = _case(None, op, B, L, H, Hkv, n, d, dtype, gen=_log(rng, 1, 200),
                  r_l=round(rng.uniform(0.0, 0.3 if n < 2000 else 0.1), 3),
                  rot=rng.choice((0, d // 2, d)), style=rng.choice(("interleaved", "half")),
                  base=rng.choice((10000.0, 500000.0)), idle=B >= 2 and rng.random() < 0.3,
                  scores=op == "shared" and rng.random() < 0.3, budget=budget, recent=recent)
        w = work(c)
        if _entries(c) * PAGE * d <= 2e8 and _gkv(c) <= 4096 and _heads(c) * n <= 1.5e8 \
                and _one(c) * n * d <= 1.2e8 and w["bytes"] <= 3e8 and w["flops"] <= 6e10 \
                and (op == "shared" or w["flops"] >= 1000):
            return c


# ------------------------------------------- what is the same for every seed
def _one(c):
    """Caches of one sequence."""
    return c["L"] * c["Hkv"]


def _gkv(c):
    return c["B"] * _one(c)


def _heads(c):
    return c["B"] * c["L"] * c["H"]


def _window(c):
    return int(math.ceil(float(np.float32(c["r_l"])) * c["n"]))


def _policies(c, count):
    """Shortlist entry of each cache: 15 % special, 20 % punct, 10 % frequent, 25 % local, 30 % full;
    sequences that share a prompt share its policies."""
    kind = (np.arange(count) % (_one(c) if c["op"] == "shared" else count) * 13 + 5) % 20
    return np.select([kind < 3, kind < 7, kind < 9, kind < 14], [S, SP, SPF, SPFL], FULL)


def _kept(c, count):
    """Never-evicted prompt rows of each cache (some special-only caches are empty)."""
    pol, n, i = _policies(c, count), c["n"], np.arange(count)
    want = np.select([pol == S, pol == SP, pol == SPF, pol == SPFL],
                     [i % 3, 1 + n // 20 + i % 7, 1 + (3 * n) // 10 + i % 17,
                      1 + (8 * n) // 25 + i % 17], n)
    return np.minimum(want, n).astype(np.int64)


def _rows(c):
    """Never-evicted rows of each sequence's own caches when the timed call begins."""
    gk = _gkv(c)
    pol = _policies(c, gk)
    grown = np.select([pol == S, pol == FULL], [0, c["gen"]], c["gen"] // 20)
    if c["op"] == "evict":  # ragged
        grown = np.maximum(0, grown - np.arange(gk) % 5 * (c["gen"] // 9))
    return grown.astype(np.int64) + (0 if c["op"] == "shared" else _kept(c, gk))


def _ring(c, count):
    return np.where(_policies(c, count) == SPFL, _window(c), 0).astype(np.int64)


def _live(c):
    """Sequences that take part (an idle one has position -1)."""
    b = np.arange(c["B"])
    return b != c["B"] - 1 if c["idle"] else b >= 0


def _entries(c):
    w = _ring(c, _gkv(c))
    return int((np.maximum(1, -(-(_rows(c) + 8) // PAGE)) + -(-w // PAGE)).sum())


# ------------------------------------------------------------------ inputs
def _inv_freq(c):
    return c["base"] ** (-np.arange(0, c["rot"], 2, dtype=np.float64) / max(c["rot"], 1))


def _values(g, shape, dtype, channels):
    """Normal values with the spread of real keys: per-cache sizes and, for keys, a few large
    channels."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((shape[0],) + (1,) * (len(shape) - 1), generator=g,
                                     device="cuda"))
    if channels:
        x[..., 3::29] *= 4.0
    return x.to(dtype)


def _pool(c, g, rows, w, policies, newest, oldest):
    """A batch of caches in use: segments of `rows` rows whose positions end before `newest` [caches],
    rings of w slots that hold the positions from `oldest` [caches] to before `newest`."""
    d, dev = c["d"], "cuda"
    seg, ring = np.maximum(1, -(-(rows + 8) // PAGE)), -(-w // PAGE)
    first = np.concatenate([[0], np.cumsum(seg + ring)[:-1]])
    entries = int((seg + ring).sum())
    desc = np.stack([policies, w, first, seg, first + seg, ring], 1).astype(np.int32)
    o = dict(caches=torch.from_numpy(desc).to(dev), rows=torch.from_numpy(rows.astype(np.int32)).to(dev),
             # pages in no particular order, as in a pool that other sequences have used
             page_table=torch.randperm(entries, generator=g, device=dev).to(torch.int32),
             next_page=torch.tensor([entries], dtype=torch.int32, device=dev),
             most=(int(seg.max()), int(ring.max())),
             k=torch.zeros((entries, PAGE, d), dtype=torch.float8_e4m3fn, device=dev),
             v=torch.zeros((entries, PAGE, d), dtype=torch.float8_e4m3fn, device=dev),
             exps=torch.full((entries, PAGE // BLOCK, 2), E_MIN, dtype=torch.int8, device=dev),
             pos=torch.full((entries, PAGE), -1, dtype=torch.int32, device=dev))
    o["rows_out"] = o["rows"].clone()
    step = 4096
    for a in range(0, entries, step):
        z = min(entries, a + step)
        for key, channels, which in (("k", True, 0), ("v", False, 1)):
            x = _values(g, (z - a, PAGE, d), torch.float32, channels).view(-1, BLOCK, d)
            ex = _exponent(x.abs().amax((1, 2)))
            o[key][a:z] = _code(x, ex[:, None, None]).view(z - a, PAGE, d)
            o["exps"][a:z, :, which] = ex.view(z - a, -1).to(torch.int8)
    newest = torch.from_numpy(newest).to(dev)[:, None]
    oldest = torch.from_numpy(oldest).to(dev)[:, None]
    # a segment's rows in order of position, the last ones the newest
    ok, at = _places(o, 2, o["most"][0])
    r = torch.arange(at.shape[1], device=dev)[None]
    ok &= r < o["rows"].long()[:, None]
    o["pos"].view(-1)[at[ok]] = (newest - o["rows"].long()[:, None] + r)[ok].clamp(min=0).to(
        torch.int32)
    # the ring's: a slot whose token went to the never-evicted segment keeps an older one, or none
    if o["most"][1]:
        wt = o["caches"][:, 1].long()[:, None]
        ok, at = _places(o, 4, o["most"][1])
        slot = torch.arange(at.shape[1], device=dev)[None]
        ok &= slot < wt
        t = newest - 1
        p = t - (t - slot) % wt.clamp(min=1)
        p = torch.where(torch.rand(p.shape, generator=g, device=dev) < 0.06, p - wt, p)
        p = torch.where(p < oldest, torch.full_like(p, -1), p)
        o["pos"].view(-1)[at[ok]] = p[ok].clamp(min=-1).to(torch.int32)
    return o


def _places(o, first, most):
    """(is there such a row, its row of the pool) for the rows of the first `most` pages of a segment
    of each cache: column `first` of caches holds its first table entry, the next its entries."""
    cc = o["caches"].long()
    j = torch.arange(most, device="cuda")[None]
    ok = j < cc[:, first + 1, None]
    page = o["page_table"].long()[torch.where(ok, cc[:, first, None] + j, 0)]
    at = page[:, :, None] * PAGE + torch.arange(PAGE, device="cuda")
    return ok.repeat_interleave(PAGE, 1), at.flatten(1)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt, G, gk, d = DTYPES[c["dtype"]], _heads(c), _gkv(c), c["d"]
    s = dict(case=c, special=torch.tensor(SPECIAL, dtype=torch.int32, device=dev),
             punct=torch.tensor(PUNCT, dtype=torch.int32, device=dev),
             dev_err=torch.zeros(1, dtype=torch.int32, device=dev))
    inv = _inv_freq(c)
    s["inv_freq"] = torch.from_numpy(inv).to(dev)
    # turns a position, as 64-bit fractions: what the framework's rotation takes
    s["turns"] = torch.tensor([int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in inv],
                              dtype=torch.int64, device=dev)
    step = c["op"] != "evict"
    at = c["n"] + c["gen"] + 3 * (np.arange(c["B"]) % 5)  # each sequence's next position
    seq = np.arange(gk) // _one(c)
    start = np.full(gk, c["n"] if c["op"] == "shared" else 0)
    s["own"] = _pool(c, g, _rows(c), _ring(c, gk), _policies(c, gk), at[seq], start)
    if c["op"] == "shared":
        m, end = _one(c), np.full(_one(c), c["n"])
        s["prompt"] = _pool(c, g, _kept(c, m), _ring(c, m), _policies(c, m), end, 0 * end)
    # a step places its token at the next position; a cut comes after one
    pos = np.where(_live(c), at - (0 if step else 1), -1).astype(np.int32)
    s["pos"] = torch.from_numpy(pos).to(dev)
    if c["scores"] or not step:
        # weights as they accumulate: a few large, many small, rows never looked at, pinned rows
        shape = (s["own"]["k"].shape[0], PAGE)
        x = torch.exp(2.0 * torch.randn(shape, generator=g, device=dev) - 3.0)
        u = torch.rand(shape, generator=g, device=dev)
        x = torch.where(u < 0.1, torch.zeros_like(x), x)
        s["scores"] = torch.where(u > 0.99, torch.full_like(x, math.inf), x)
    if step:
        ids = torch.randint(2, 32000, (c["B"],), generator=g, device=dev, dtype=torch.int32)
        pick = torch.rand(c["B"], generator=g, device=dev)
        ids = torch.where(pick < 0.1, s["punct"][(ids % len(PUNCT)).long()], ids)
        s["ids"] = torch.where(pick > 0.95, torch.full_like(ids, SPECIAL[0]), ids)
        s["q"] = _values(g, (G, d), dt, False)
        s["k_new"], s["v_new"] = _values(g, (gk, d), dt, True), _values(g, (gk, d), dt, False)
        s["out"] = torch.zeros((G, d), dtype=dt, device=dev)
    if own:
        _handles(s)
    return s


# ------------------------------------------------------------ the framework
def _handles(s):
    from adaptive_head_kv_gb300 import fastgen as fg

    c = s["case"]
    code = {"bf16": fg.FG_BF16, "fp32": fg.FG_FP32}[c["dtype"]]

    def params(B):
        return fg.Params(B, c["L"], c["H"], c["n"], c["d"], code, 0.95, c["r_l"], 0.3, 0.0,
                         c["Hkv"])

    def cache(p, o):
        return fg.PagedCache(p, o["k"], o["v"], o["exps"], o["pos"], o["page_table"], o["caches"],
                             o["rows"], o["next_page"], rows_out=o["rows_out"])

    s["p"] = params(c["B"])
    s["cache"] = cache(s["p"], s["own"])
    s["prefix"] = cache(params(1), s["prompt"]) if c["op"] == "shared" else None
    s["rope"] = None
    if c["rot"]:
        s["rope"] = fg.Rope(s["turns"], style={"interleaved": fg.FG_ROPE_INTERLEAVED,
                                               "half": fg.FG_ROPE_HALF}[c["style"]])
    if c["op"] == "evict":
        need = fg.fastgen_evict_q8_workspace_bytes(s["p"], c["budget"])
    else:
        s["cache"].schedule(s["p"])
        need = fg.fastgen_decode_q8_ex_workspace_bytes(s["p"], s["cache"], s["prefix"],
                                                       c["scores"])
    s["ws"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")


def _run_own(s):
    from adaptive_head_kv_gb300 import fastgen as fg

    c = s["case"]
    if c["op"] == "evict":
        fg.fastgen_evict_q8(s["p"], s["cache"], s["scores"], c["budget"], c["recent"], s["pos"],
                            s["ws"], s["dev_err"])
    else:
        fg.fastgen_decode_attn_q8_ex(s["p"], s["cache"], s["prefix"], s.get("scores"), s["q"],
                                     s["k_new"], s["v_new"], s["ids"], s["special"], s["punct"],
                                     s["pos"], s["rope"], s["out"], s["ws"], s["dev_err"])


def run(state):
    s = state
    if own:
        _run_own(s)
    elif s["case"]["op"] == "evict":
        _evict_plain(s)
    else:
        _step_plain(s)
    o = {key: s["own"][key] for key in ("k", "v", "exps", "pos")}
    o["rows"] = s["own"]["rows_out"]
    for key in ("scores", "out"):
        if key in s:
            o[key] = s[key]
    return o


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


def _write_rows(o, at, xk, xv, fresh):
    """Codes rows xk, xv [r, d] into pool rows `at` [r]; fresh [r]: the row's block starts anew.
    Other rows of a block whose exponent grows are rounded again."""
    d = o["k"].shape[-1]
    blocks, nb = at // BLOCK, o["k"].shape[0] * (PAGE // BLOCK)
    touched = torch.zeros(nb, dtype=torch.bool, device="cuda")
    touched[blocks] = True
    anew = torch.zeros(nb, dtype=torch.bool, device="cuda")
    anew[blocks] = fresh
    ids = touched.nonzero()[:, 0]
    for key, x, which in (("k", xk, 0), ("v", xv, 1)):
        need = torch.full((nb,), -128, dtype=torch.int32, device="cuda")
        need.scatter_reduce_(0, blocks, _exponent(_amax(x, -1)), "amax")
        had = o["exps"].view(nb, 2)[:, which].int()
        had = torch.where(anew, torch.full_like(had, -128), had)
        now = torch.maximum(need, had)
        codes = o[key].view(torch.uint8).view(nb, BLOCK, d)
        shift = torch.where(anew, torch.zeros_like(now), had - now)[ids]
        old = codes[ids].view(torch.float8_e4m3fn).float()
        codes[ids] = (old * _pow2(shift).float()[:, None, None]).to(torch.float8_e4m3fn).view(
            torch.uint8)
        o[key].view(torch.uint8).view(-1, d)[at] = _code(x, now[blocks][:, None]).view(torch.uint8)
        o["exps"].view(nb, 2)[:, which][ids] = now[ids].to(torch.int8)


def _values_of(o, key, at):
    """Rows `at` of the pool in 32 bits."""
    d = o["k"].shape[-1]
    x = o[key].view(torch.uint8).view(-1, d)[at].view(torch.float8_e4m3fn).float()
    e = o["exps"].view(-1, 2)[:, 0 if key == "k" else 1].int()[at // BLOCK]
    return x * _pow2(e).float()[..., None]


def _append_plain(s):
    """The step's token into each cache."""
    c, o = s["case"], s["own"]
    seq = torch.arange(_gkv(c), device="cuda") // _one(c)
    cc, table = o["caches"].long(), o["page_table"].long()
    special = (s["ids"][:, None] == s["special"]).any(-1)
    punct = (s["ids"][:, None] == s["punct"]).any(-1)
    pol, w, rows = cc[:, 0], cc[:, 1], o["rows"].long()
    to_segment = (pol == FULL) | special[seq] | ((pol != S) & punct[seq])
    pos = s["pos"].long()[seq]
    st = to_segment & (pos >= 0) & (rows < cc[:, 3] * PAGE)
    ring = ~to_segment & (pos >= 0) & (pol == SPFL) & (w > 0)
    place = torch.where(st, rows, pos % w.clamp(min=1))
    put = st | ring
    entry = torch.where(st, cc[:, 2], cc[:, 4]) + place // PAGE
    at = table[torch.where(put, entry, 0)] * PAGE + place % PAGE
    k = _rotated(s["k_new"], pos, c, s["inv_freq"])
    _write_rows(o, at[put], k[put], s["v_new"].float()[put], (st & (rows % BLOCK == 0))[put])
    o["pos"].view(-1)[at[put]] = pos[put].to(torch.int32)
    o["rows_out"].copy_((rows + st).to(torch.int32))
    if "scores" in s:
        first = torch.where(special[seq], math.inf, 0.0).float()
        s["scores"].view(-1)[at[st]] = first[st]


def _rows_of(o, key_rows, t):
    """Of each cache: which rows of its segment are there, which slots of its ring, which of those
    each sequence sees at t [.., caches or 1, 1], and all their rows of the pool."""
    a, pa = _places(o, 2, o["most"][0])
    row = torch.arange(pa.shape[1], device="cuda")[None]
    a &= row < o[key_rows].long()[:, None]
    b, pb = _places(o, 4, o["most"][1])
    slot = torch.arange(pb.shape[1], device="cuda")[None]
    w, p = o["caches"][:, 1].long()[:, None], o["pos"].view(-1)[pb].long()
    b = b & (slot < w) & (p >= 0)
    near = (p > t - w) & (p <= t)
    return a, b, near, torch.cat([pa, pb], 1)


def _step_plain(s):
    _append_plain(s)
    c, o, d = s["case"], s["own"], s["case"]["d"]
    B, m, R = c["B"], _one(c), c["H"] // c["Hkv"]
    t = s["pos"].long()
    seq = torch.arange(B * m, device="cuda") // m
    mine, b, near, at = _rows_of(o, "rows_out", t[seq][:, None])
    ok = torch.cat([mine, b & near], 1).view(B, m, 1, -1)
    q = _rotated(s["q"].view(B, -1, d), t.clamp(min=0)[:, None], c, s["inv_freq"])
    q = q.view(B, m, R, d) / math.sqrt(d)
    k = _values_of(o, "k", at).view(B, m, -1, d)
    score = torch.matmul(q, k.transpose(2, 3)).masked_fill(~ok, -math.inf)
    top = score.amax(-1, keepdim=True)
    if "prompt" in s:
        o = s["prompt"]
        a, b, near, pat = _rows_of(o, "rows", t[:, None, None])
        there = torch.cat([a[None].expand(B, -1, -1), b & near], 2)[:, :, None]
        # one product for all sequences: [caches, B * R, d] with [caches, d, rows]
        k = _values_of(o, "k", pat)
        ps = torch.matmul(q.transpose(0, 1).reshape(m, B * R, d), k.transpose(1, 2))
        ps = ps.view(m, B, R, -1).transpose(0, 1).masked_fill(~there, -math.inf)
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    if "prompt" in s:
        pe = torch.exp(ps - top)
        total = total + pe.sum(-1, keepdim=True)
    e = e / total.clamp(min=1e-30)
    v = _values_of(s["own"], "v", at).view(B, m, -1, d).masked_fill(~ok.transpose(2, 3), 0.0)
    out = torch.matmul(e, v)
    if "prompt" in s:
        pe = (pe / total.clamp(min=1e-30)).transpose(0, 1).reshape(m, B * R, -1)
        v = _values_of(o, "v", pat).masked_fill(~torch.cat([a, b], 1)[..., None], 0.0)
        out = out + torch.matmul(pe, v).view(m, B, R, d).transpose(0, 1)
    active = (t >= 0)[:, None, None, None]
    s["out"].copy_(torch.where(active, out, s["out"].view(B, m, R, d).float()).view(-1, d))
    if "scores" in s:
        live, seg = mine & (t >= 0)[seq][:, None], mine.shape[1]
        w = e.sum(2).view(B * m, -1)[:, :seg]
        s["scores"].view(-1)[at[:, :seg][live]] += w[live]


def _evict_plain(s):
    c, o = s["case"], s["own"]
    seq = torch.arange(_gkv(c), device="cuda") // _one(c)
    rows, t, budget = o["rows"].long()[:, None], s["pos"].long()[seq][:, None], c["budget"]
    cut = ((rows > budget) & (t >= 0))[:, 0]
    ok, at = _places(o, 2, o["most"][0])
    r = torch.arange(at.shape[1], device="cuda")[None]
    ok = ok & (r < rows) & cut[:, None]
    p = o["pos"].view(-1)[at].long()
    score = s["scores"].view(-1)[at]
    score = torch.where(score > 0, score, torch.zeros_like(score))
    key = score.view(torch.int32).long()
    key = torch.where((p > t - c["recent"]) & (p <= t), torch.full_like(key, 0x7FFFFFFF), key)
    key = torch.where(ok, (key << 32) - r, torch.full_like(key, -(1 << 62)))
    if at.shape[1] > budget:
        least = key.sort(1, descending=True)[0][:, budget - 1, None]
        hole = (ok & (key < least) & (r < budget)).nonzero(as_tuple=True)
        mover = (ok & (key >= least) & (r >= budget)).nonzero(as_tuple=True)
        to, fr = at[hole], at[mover]
        k, v = _values_of(o, "k", fr), _values_of(o, "v", fr)
        _write_rows(o, to, k, v, torch.zeros_like(to, dtype=torch.bool))
        for x in (o["pos"], s["scores"]):
            x.view(-1)[to] = x.view(-1)[fr]
    o["rows_out"].copy_(torch.where(cut, torch.full_like(rows[:, 0], budget), rows[:, 0]).to(
        torch.int32))


# ----------------------------------------------------------------- the work
def work(case):
    c = case
    eb = 2 if c["dtype"] == "bf16" else 4
    d, R, m = c["d"], c["H"] // c["Hkv"], _one(c)
    live = np.repeat(_live(c), m)
    rows, w = _rows(c), _ring(c, _gkv(c))
    if c["op"] == "evict":
        over = np.where(live & (rows > c["budget"]), rows, 0)
        cut = over > 0
        # the newest rows, a share of the others by weight, come from behind the budget
        moved = float(np.minimum(np.where(cut, rows - c["budget"], 0), c["budget"]).sum()) * 0.6
        return dict(bytes=8.0 * over.sum() + moved * (4 * d + 16) + 8 * _gkv(c),
                    flops=4.0 * over.sum() + 4 * moved * d)
    # of a ring that began with the prompt's end only the slots written since are there
    ring = np.minimum(w, c["gen"]) if c["op"] == "shared" else w
    att = float(((rows + ring) * live).sum())
    nl = float(live.sum())
    bytes_ = att * 2 * d + att / 8 + 4 * float((ring * live).sum()) + nl * (2 * R + 4) * eb * d
    flops = 4 * R * att * d + 3 * nl * (R + 1) * c["rot"]
    if c["scores"]:
        bytes_ += 8 * float((rows * live).sum())
        flops += R * float((rows * live).sum())
    if c["op"] == "shared":
        prompt = float((_kept(c, m) + _ring(c, m)).sum())
        bytes_ += prompt * 2 * d + prompt / 8 + 4 * float(_ring(c, m).sum())
        flops += 4 * R * prompt * d * float(_live(c).sum())
    return dict(bytes=bytes_, flops=flops)


# ---------------------------------------------------- the definition, 64 bits
def _nearest_code(y):
    """Nearest e4m3 value of y (numpy, 64 bits): three fraction bits, exponents from -6."""
    a = np.minimum(np.abs(y), CODE_MAX)
    step = np.ldexp(1.0, np.maximum(np.frexp(a)[1] - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, CODE_MAX), y)


def _least_exponents(amax):
    f, e = np.frexp(amax / CODE_MAX)
    return np.maximum(np.where(amax > 0, np.where(f == 0.5, e - 1, e), E_MIN), E_MIN)


def _turn(x, p, c):
    """Rows x [r, d] at positions p [r], rotated in 64 bits."""
    x, rot = np.array(x, dtype=np.float64), c["rot"]
    z = np.exp(1j * np.multiply.outer(np.asarray(p, dtype=np.float64), _inv_freq(c)))
    i, j = ((slice(0, rot // 2), slice(rot // 2, rot)) if c["style"] == "half" else
            (slice(0, rot, 2), slice(1, rot, 2)))
    u = (x[:, i] + 1j * x[:, j]) * z
    x[:, i], x[:, j] = u.real, u.imag
    return x


class _Host:
    """A batch of caches on the host, in 64 bits."""

    def __init__(self, o):
        self.k, self.v = (o[x].double().cpu().numpy().reshape(-1, o[x].shape[-1]) for x in "kv")
        self.e = o["exps"].cpu().numpy().astype(np.int64).reshape(-1, 2)
        self.p = o["pos"].cpu().numpy().astype(np.int64).reshape(-1)
        self.caches = o["caches"].cpu().numpy().astype(np.int64)
        self.table = o["page_table"].cpu().numpy().astype(np.int64)
        self.rows = o["rows"].cpu().numpy().astype(np.int64)

    def seg(self, i, rows):
        return self.table[self.caches[i, 2] + rows // PAGE] * PAGE + rows % PAGE

    def ring(self, i, slots):
        return self.table[self.caches[i, 4] + slots // PAGE] * PAGE + slots % PAGE

    def value(self, side, at):
        return (self.k, self.v)[side][at] * 2.0 ** self.e[at // BLOCK, side][:, None]

    def put(self, at, keys, values, anew):
        """Rows into the pool, one block after the other."""
        for b in np.unique(at // BLOCK):
            i = np.flatnonzero(at // BLOCK == b)
            whole = slice(b * BLOCK, (b + 1) * BLOCK)
            for side, (pool, x) in enumerate(((self.k, keys[i]), (self.v, values[i]))):
                now = int(_least_exponents(np.abs(x).max(1)).max())
                if not anew[i[0]]:
                    now = max(now, self.e[b, side])
                    pool[whole] = _nearest_code(pool[whole] * 2.0 ** float(self.e[b, side] - now))
                pool[at[i]] = _nearest_code(x * 2.0 ** -float(now))
                self.e[b, side] = now


def exact(case, seed):
    c = case
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    h = _Host(s["own"])
    pos = s["pos"].cpu().numpy().astype(np.int64)
    score = s["scores"].double().cpu().numpy().reshape(-1) if "scores" in s else None
    o = dict(exps=None, pos=None, rows=None)
    if c["op"] == "evict":
        _exact_cut(c, h, pos, score)
    else:
        ids = s["ids"].cpu().numpy()
        pinned = np.isin(ids, SPECIAL)
        seg = []  # each cache's segment rows in the pool, the new one among them
        put = []
        for i, (pol, w, _, cap, _, _) in enumerate(h.caches):
            b = i // _one(c)
            rows = h.rows[i]
            if pos[b] >= 0 and (pol == FULL or pinned[b] or (pol != S and ids[b] in PUNCT)):
                if rows < cap * PAGE:
                    at = int(h.seg(i, rows))
                    put.append((i, at, rows % BLOCK == 0))
                    rows += 1
                    if score is not None:
                        score[at] = math.inf if pinned[b] else 0.0
            elif pos[b] >= 0 and pol == SPFL and w > 0:
                put.append((i, int(h.ring(i, pos[b] % w)), False))
            seg.append(h.seg(i, np.arange(rows)))
        if put:
            i, at, anew = (np.array(x) for x in zip(*put))
            p = pos[i // _one(c)]
            k, v = (s[x].double().cpu().numpy()[i] for x in ("k_new", "v_new"))
            h.put(at, _turn(k, p, c), v, anew)
            h.p[at] = p
        o["out"] = _exact_attend(c, s, h, pos, seg, score)
    shape = tuple(s["own"]["k"].shape)
    o["k"], o["v"] = (torch.from_numpy(x).view(shape) for x in (h.k, h.v))
    if score is not None:
        o["scores"] = torch.from_numpy(score).view(shape[:2])
    return o


def _exact_cut(c, h, pos, score):
    for i, rows in enumerate(h.rows):
        t = pos[i // _one(c)]
        if t < 0 or rows <= c["budget"]:
            continue
        at = h.seg(i, np.arange(rows))
        near = (h.p[at] > t - c["recent"]) & (h.p[at] <= t)
        weight = np.where(score[at] > 0, score[at], 0.0)
        kept = np.sort(np.lexsort((np.arange(rows), -weight, ~near))[: c["budget"]])
        hole = np.setdiff1d(np.arange(c["budget"]), kept)
        mover = kept[kept >= c["budget"]]
        to, fr = at[hole], at[mover]
        h.put(to, h.value(0, fr), h.value(1, fr), np.zeros(len(to), dtype=bool))
        h.p[to], score[to] = h.p[fr], score[fr]


def _exact_attend(c, s, h, pos, seg, score):
    """Attention of every sequence, one cache of a sequence's set after the other, on the GPU."""
    R, d, m, B = c["H"] // c["Hkv"], c["d"], _one(c), c["B"]
    q = s["q"].double().cpu().numpy()
    q = _turn(q, np.repeat(pos.clip(min=0), len(q) // B), c).reshape(B, m, R, d)
    both = [(h, torch.from_numpy(h.k).cuda(), torch.from_numpy(h.v).cuda())]
    if "prompt" in s:
        p = _Host(s["prompt"])
        both.append((p, torch.from_numpy(p.k).cuda(), torch.from_numpy(p.v).cuda()))

    def part(which, at):
        x, k, v = both[which]
        z = torch.from_numpy(at).cuda()
        e = torch.from_numpy(2.0 ** x.e[at // BLOCK]).cuda()
        return k[z] * e[..., :1], v[z] * e[..., 1:]

    def slots(x, i, b):
        w = x.caches[i, 1]
        at = x.ring(i, np.arange(w)) if w else np.zeros(0, dtype=np.int64)
        p = x.p[at]
        return at, (p >= 0) & (p > pos[b] - w) & (p <= pos[b])

    out = torch.zeros((B, m, R, d), dtype=torch.float64, device="cuda")
    for i in range(m):
        qi = torch.from_numpy(q[:, i]).cuda()
        if "prompt" in s:
            at, _ = slots(both[1][0], i, 0)
            fixed = both[1][0].seg(i, np.arange(both[1][0].rows[i]))
            pk, pv = part(1, np.concatenate([fixed, at]))
            see = np.stack([np.concatenate([np.ones(len(fixed), bool), slots(both[1][0], i, b)[1]])
                            for b in range(B)])
            ps = (qi.view(B * R, d) @ pk.T / math.sqrt(d)).view(B, R, -1)
            ps = ps.masked_fill(~torch.from_numpy(see).cuda()[:, None], -math.inf)
        mine = []
        for b in range(B):
            at, ok = slots(h, b * m + i, b)
            mine.append(np.concatenate([seg[b * m + i], at[ok]]))
        most = max(len(x) for x in mine)
        at = np.stack([np.pad(x, (0, most - len(x))) for x in mine])
        there = np.arange(most)[None] < np.array([len(x) for x in mine])[:, None]
        k, v = part(0, at)
        sc = torch.einsum("brd,bnd->brn", qi, k) / math.sqrt(d)
        sc = sc.masked_fill(~torch.from_numpy(there).cuda()[:, None], -math.inf)
        if "prompt" in s:
            sc = torch.cat([sc, ps], -1)
        if sc.shape[-1] == 0:
            continue
        wt = torch.softmax(sc, -1).nan_to_num(0.0)  # no row at all: zeros
        y = torch.einsum("brn,bnd->brd", wt[..., :most], v)
        if "prompt" in s:
            y = y + (wt[..., most:].reshape(B * R, -1) @ pv).view(B, R, d)
        live = torch.from_numpy(pos >= 0).cuda()
        out[:, i] = torch.where(live[:, None, None], y, out[:, i])
        if score is not None:
            got = wt[..., :most].sum(1).cpu().numpy()
            for b in range(B):
                if pos[b] >= 0:
                    score[seg[b * m + i]] += got[b, : len(seg[b * m + i])]
    return out.view(-1, d).cpu()
