"""What the cut to a budget promises: which rows a pinned one gives way to."""
import pytest
import torch

import paged_ref as P
from adaptive_head_kv_gb300 import fastgen as fg
from test_paged_gpu import dev, gen
from test_paged_step_gpu import Step

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
