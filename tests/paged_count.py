"""Caches that show each of their rows: every query is zero, so that all live
rows weigh the same, and a row's values are one 1 at a dimension given by its
position.  An output is then the number of live rows of each dimension over
the number of all, and one row too few or too many moves a value by more than
any rounding."""
import numpy as np
import torch

import paged_ref as P


class Positions(P.RefCache):
    """Which positions a cache holds (no keys, no values)."""

    def __init__(self, policy, w, cap, d):
        self.policy, self.w, self.cap, self.d = policy, w if policy == P.SPFL else 0, cap, d
        self.rows, self.seg, self.ring = 0, {}, {}
        self.seg_pos, self.ring_pos = np.full(cap, -1), np.full(self.w, -1)

    def compact(self, static, window, K=None, V=None):
        self.rows = len(static)
        self.seg_pos[: self.rows] = static
        for j in window:
            self.ring_pos[j % self.w] = j

    def append(self, k, v, kinds, pos, room=None):
        for i, kind in enumerate(kinds):
            if self.to_segment(*kind):
                if self.rows < self.cap:
                    self.seg_pos[self.rows] = pos + i
                    self.rows += 1
            elif self.w and i >= len(kinds) - self.w:
                self.ring_pos[(pos + i) % self.w] = pos + i

    def positions(self, t):
        a, b = self.live(t)
        return np.concatenate([self.seg_pos[a], self.ring_pos[b]]).astype(int)


def dimension(pos, d, step):
    """Blocks of 16 positions at a dimension (step 0), or single ones scattered over all."""
    return (pos // 16 if step == 0 else (pos.astype(np.int64) * 2654435761 >> 13)) % d


def values(pos, d, step):
    v = torch.zeros(*pos.shape, d)
    v.scatter_(-1, torch.as_tensor(dimension(np.asarray(pos), d, step))[..., None], 1.0)
    return v


def counts(pos, d, step):
    return np.bincount(dimension(pos, d, step), minlength=d) / max(len(pos), 1)


def bound(want, dtype):
    """Weights within 2^-10 (two f16 terms or one, sums in 32 bits), the result rounded to its
    type."""
    return np.abs(want) * (2.0 ** -10 + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)) + 1e-12
