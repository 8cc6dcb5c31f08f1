"""The counting caches' bound sees every row: one missing, or one twice, passes it."""
import numpy as np
import pytest

import paged_count as C
import paged_ref as P


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 17, 333, 1300, 2600, 4200])
@pytest.mark.parametrize("step", [0, 1])
def test_a_row_or_a_block_too_few_or_too_many_passes_the_bound(n, d, step):
    pos = np.arange(n)
    want = C.counts(pos, d, step)
    bound = C.bound(want, "bf16")
    for first in (0, n // 2, n - 1):  # a row, a block of 16, a page; missing or twice
        for rows in (1, 16, 64):
            some = pos[first: first + rows]
            if len(some) == n:
                continue
            less, more = np.setdiff1d(pos, some), np.concatenate([pos, some])
            assert (np.abs(C.counts(less, d, step) - want) > bound).any()
            assert (np.abs(C.counts(more, d, step) - want) > bound).any()


def test_positions_are_the_reference_caches():
    rng = np.random.default_rng(1)
    for policy in range(5):
        a, b = P.RefCache(policy, 13, 256, 64), C.Positions(policy, 13, 256, 64)
        n = 40
        static = [j for j in range(n) if policy == P.FULL or rng.random() < 0.2]
        window = [j for j in range(n - 13, n) if j not in static] if policy == P.SPFL else []
        K = rng.normal(size=(n, 64))
        for c in (a, b):
            c.compact(static, window, K, K)
        t = n
        for m in (1, 5, 30, 1, 20):
            kinds = [(rng.random() < 0.1, rng.random() < 0.2) for _ in range(m)]
            rows = rng.normal(size=(m, 64))
            for c in (a, b):
                c.append(rows, rows, kinds, t)
            t += m
            assert a.rows == b.rows and np.array_equal(a.seg_pos[: a.rows], b.seg_pos[: b.rows])
            assert np.array_equal(a.ring_pos, b.ring_pos)
            assert all(np.array_equal(x, y) for x, y in zip(a.live(t - 1), b.live(t - 1)))
