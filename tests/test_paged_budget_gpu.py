"""What the cut to a budget promises: which rows a pinned one gives way to, what becomes of it in a
step of NaN, and the pages that a long generation needs."""
import pytest
import torch

import paged_ref as P
from adaptive_head_kv_gb300 import fastgen as fg
from adaptive_head_kv_gb300.session import PagedSession, make_params
from test_paged_gpu import PUNCT, SPECIAL, dev, gen
from test_paged_step_gpu import Step, check_cut

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget,recent", [(48, 16), (32, 16), (32, 31), (32, 32)])
def test_pinned_rows_rank_behind_recent_ones_alone(budget, recent):
    """20 rows with +inf among 200: they stay, lower rows first, as far as the recent rows leave
    room, and before any other row."""
    n, pinned = 200, list(range(3, 43, 2))
    s = Step(61, L=1, H=2, n=n, policies=[4])
    s.compact()
    weights = torch.rand(s.cache.c.n_pages, 64, generator=gen(1)) + 1.0
    gpu = P.GpuPages(s.cache)
    for c in range(s.gk):
        pages = gpu.pages(c, False)
        for r in pinned:
            weights[int(pages[r // 64]), r % 64] = float("inf")
    s.scores = dev(weights)
    ws = torch.empty(fg.fastgen_evict_q8_workspace_bytes(s.p, budget), dtype=torch.uint8,
                     device="cuda")
    fg.fastgen_evict_q8(s.p, s.cache, s.scores, budget, recent, dev([n - 1], torch.int32), ws, s.err)
    assert int(s.err.item()) == 0 and s.cache.rows.tolist() == [budget] * s.gk
    after = P.GpuPages(s.cache)
    left = budget - recent
    for c in range(s.gk):
        # (a full cache's rows are its positions)
        stay = set(after.segment(c, False, budget)["pos"].tolist())
        want = set(range(n - recent, n)) | set(pinned[:left])
        rest = [r for r in range(n - recent) if r not in pinned]
        w = weights[torch.as_tensor(gpu.pages(c, False).repeat(64)[:n]), torch.arange(n) % 64]
        want |= set(sorted(rest, key=lambda r: (-float(w[r]), r))[: max(0, left - len(pinned))])
        assert stay == want


@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1)])
def test_a_step_with_nan_leaves_pinned_rows_pinned(H, Hkv):
    """Weights that are NaN make the rows' scores NaN, which count as 0 from then on, but not those
    of special tokens."""
    s = Step(62, L=1, H=H, Hkv=Hkv, n=150, policies=[4]).with_scores(2)
    s.compact()
    before = s.scores.clone()
    q = torch.randn(s.G, s.d, generator=gen(1))
    q[1] = float("nan")
    s.decode(q.to(torch.bfloat16), None, None, None, [150])
    gpu, sick = P.GpuPages(s.cache), 1 // s.R
    for c in range(s.gk):
        at = torch.as_tensor(gpu.pages(c, False)[:3])
        was, now = (x[at.cuda()].reshape(-1)[:150] for x in (before, s.scores))
        pinned = torch.isinf(was)
        assert pinned.any() and torch.equal(torch.isinf(now), pinned)
        assert bool(torch.isnan(now[~pinned]).all()) == (c == sick)


@pytest.mark.parametrize("forked", [False, True])
def test_a_long_generation_within_the_pages_of_a_budget(forked):
    """Room for budget + 16 new rows a cache and a cut every 16 steps: any number of steps, with the
    results that room for all of them gives; without cuts that room ends, and a step says so."""
    L, H, n, d, budget, every, steps = 1, 4, 150, 64, 48, 16, 120
    B = 2 if forked else 1
    p = make_params(1, L, H, n, d, "bf16", 0.9, 0.3, 0.3)
    g = gen(63)
    Q, K, V = (dev(torch.randn(H, n, d, generator=g).to(torch.bfloat16)) for _ in range(3))
    ids = dev(torch.randint(100, 300, (1, n), generator=g, dtype=torch.int32))
    q = dev(torch.randn(steps, 3, B * H, d, generator=g).to(torch.bfloat16))
    new = dev(torch.randint(100, 300, (steps, B), generator=g, dtype=torch.int32))
    full = torch.full((H,), 4, dtype=torch.int8)

    def generate(room, cuts):
        s = PagedSession(p, SPECIAL, PUNCT, 1 if forked else room, budget=0 if forked else budget,
                         recent=0 if forked else 8)
        s.prefill_with_policy(Q, K, V, ids, full)
        if forked:
            s = s.fork(B, room, budget=budget, recent=8)
        elif cuts:
            s.evict(n - 1)
        outs, held = [], s.cache.c.n_pages
        for st in range(steps):
            outs.append(s.decode(*q[st], new[st], n + st).clone())
            if cuts and st % every == every - 1:
                s.evict(n + st)
        return s, torch.stack(outs), held, fg.fastgen_read_error(s.dev_err)

    s, outs, held, err = generate(budget + every, True)
    assert err == fg.FG_OK and (s.cache.rows <= budget + every).all()
    # a fork's caches begin empty, a prompt's with all of its rows
    assert held == s.Gkv * -(-(budget + every + (0 if forked else n)) // 64)
    wide, want, more, err = generate(steps, True)
    assert err == fg.FG_OK and more > held and torch.equal(outs, want)
    assert torch.equal(s.cache.rows, wide.cache.rows)
    assert generate(budget + every, False)[3] == fg.FG_ECAPACITY


@pytest.mark.parametrize("n,policies,recent", [
    (4500, [4, 2, 1, 3, 0, 1], 100),  # long caches among short ones: room for 0.3 of the prompt
    (4500, [4] + [0] * 31, 0),        # one of 32: room for less than an eighth
    (4090, [4, 0, 3], 4000),
])
def test_cut_of_caches_of_many_lengths(n, policies, recent):
    """Some caches hold more rows than the small form has places for, the others few."""
    s = Step(64, L=1, H=len(policies), n=n, d=64, policies=policies, max_new=4).with_scores(5)
    s.compact()
    assert check_cut(s, 4000, recent, [n - 1]) > 0
    assert sorted(set(s.cache.rows.tolist()))[-1] == 4000 < n
    s.check()
    assert int(s.err.item()) == 0
