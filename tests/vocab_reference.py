"""The embedding, its gradient, the step of beam search and the reordering of
states in float64 numpy, from their definitions, with the error bounds that the
GPU tests hold results to. Shares no code with the library."""
from __future__ import annotations

import numpy as np

from ops_reference import HALF, U

TINY = 2.0 ** -133   # half a step of bf16's smallest values; float32's is smaller


def embed(W, ids, scale, y_type):
    """y and its largest errors: W widened is exact, one product in float32, one rounding when stored."""
    V = W.shape[0]
    live = (ids >= 0) & (ids < V)
    s = np.float64(np.float32(scale))
    y = np.where(live[:, None], W.astype(np.float64)[np.where(live, ids, 0)] * s, 0.0)
    e = np.abs(y) * U
    return y, np.where(live[:, None], e * (1 + HALF[y_type]) + HALF[y_type] * np.abs(y) + TINY, 0.0)


def embed_grad(ids, dy, V, scale, old, g_type):
    """dW and its largest errors; `old` is what it is added to, or None. A word's n rows take n additions, its scale
    a product and (added) a sum."""
    live = (ids >= 0) & (ids < V)
    s = np.float64(np.float32(scale))
    dy = dy.astype(np.float64)[live]
    total, size = (np.zeros((V, dy.shape[1])) for _ in range(2))
    np.add.at(total, ids[live], dy)
    np.add.at(size, ids[live], np.abs(dy))
    n = np.bincount(ids[live], minlength=V)[:, None]
    dW = s * total
    e = np.abs(s) * size * (n + 1) * U
    if old is not None:
        dW = dW + old.astype(np.float64)
        e = e + U * (np.abs(dW) + e)
    e = e * (1 + HALF[g_type]) + HALF[g_type] * np.abs(dW) + TINY
    return dW, np.where(n > 0, e, 0.0)   # rows without a token are exact


class Beams:
    """Every candidate's score of one step: `found` [N, V], -inf where there is none."""

    def __init__(self, h, W, scores, beams, C, ended=None, allowed=None, T=1.0):
        h, W = h.astype(np.float64), W.astype(np.float64)
        N, V = len(h), len(W)
        self.V, self.G, self.C = V, beams, C
        s = scores.astype(np.float64)
        out = np.zeros(N, bool) if ended is None else (ended >= 0) & (ended < V)
        part = np.isfinite(s)
        with np.errstate(all="ignore"):
            z = np.where((part & ~out)[:, None], h, 0.0) @ W.T / T
            m = z.max(1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
            lse = np.where(np.isposinf(z).any(1) & ~np.isnan(z).any(1), np.inf, lse)
            found = s[:, None] + (z - lse[:, None])
        self.lse = np.where(part & ~out, lse, 0.0)
        found = np.where((part & np.isfinite(lse))[:, None] & ~np.isnan(found), found, -np.inf)
        if allowed is not None:
            v = np.arange(V)
            bits = (allowed.view(np.uint32)[:, v >> 5] >> (v & 31).astype(np.uint32)) & 1
            found = np.where(bits != 0, found, -np.inf)
        for r in np.flatnonzero(out):
            found[r] = -np.inf
            if part[r]:
                found[r, ended[r]] = s[r]
        self.found = found
        flat = found.reshape(N // beams, beams * V)
        flat = np.pad(flat, ((0, 0), (0, C)), constant_values=-np.inf)   # there may be fewer words than candidates
        order = np.argsort(-flat, axis=1, kind="stable")[:, :C]   # equal ones: the lowest row, then the lowest word
        self.top = np.take_along_axis(flat, order, 1)
        first = beams * np.arange(N // beams)[:, None]
        none = np.isneginf(self.top)
        self.ids = np.where(none, -1, order % V)
        self.parents = np.where(none, -1, order // V + first)
        # a float32 logit is H products and sums off at most (its exponentials' and their sum's roundings beside it):
        # what lse is off; of the scores' order, only lse's part of that counts
        with np.errstate(all="ignore"):
            finite = [np.where(np.isfinite(x), np.abs(x), 0.0) for x in (h, W)]
            mag = (finite[0] @ finite[1].T).max(1) / T
            self.e_lse = (h.shape[1] + 8) * U * mag + (2 ** 10 + 8) * U + 8 * U * (np.abs(lse) + mag)
        self.e_lse = np.where(np.isfinite(self.lse) & np.isfinite(self.e_lse), self.e_lse, 0.0)

    def check(self, scores, ids, parents, lse, what, exactly=False):
        """The outputs against the definition. `exactly`: words and parents have to be the same ones (cases without
        near ties); otherwise each has to be within what lse is off of the score at its place, and none may occur twice."""
        lim = np.repeat(self.e_lse.reshape(-1, self.G).max(1)[:, None], self.C, 1)
        top = self.top
        assert np.array_equal(np.isneginf(scores), np.isneginf(top)), f"{what}: another number of candidates"
        none = np.isneginf(top)
        assert (ids[none] == -1).all() and (parents[none] == -1).all(), what
        with np.errstate(all="ignore"):
            off = np.where(none, 0.0, np.abs(scores - np.where(none, 0.0, top)))
            bound = lim + U * np.abs(np.where(none, 0.0, top))
        assert (off <= bound).all(), (what, off.max(), bound.min())
        if exactly:
            assert np.array_equal(ids, self.ids), (what, np.argwhere(ids != self.ids)[:4])
            assert np.array_equal(parents, self.parents), (what, np.argwhere(parents != self.parents)[:4])
        b = np.broadcast_to(np.arange(len(top))[:, None], top.shape)
        there = ~none
        assert (parents[there] // self.G == b[there]).all(), f"{what}: a parent of another group"
        at = self.found[parents[there], ids[there]]
        assert (np.abs(at - top[there]) <= 2 * lim[there]).all(), (what, np.abs(at - top[there]).max())
        flat = parents[there].astype(np.int64) * self.V + ids[there]
        assert len(np.unique(flat)) == len(flat), f"{what}: a candidate twice"
        fine = np.isfinite(self.lse)
        assert np.array_equal(np.isnan(lse), np.isnan(self.lse)) and np.array_equal(lse[~fine & ~np.isnan(lse)], self.lse[~fine & ~np.isnan(self.lse)]), what
        assert (np.abs(lse[fine] - self.lse[fine]) <= (self.e_lse + U * np.abs(self.lse))[fine]).all(), (what, "lse")
        assert (lse[self.lse == 0] == 0).all(), what


def reorder(states, out, parents, beams, lengths=None, row_dim=0, length_dim=None):
    """What out holds afterwards."""
    got = out.copy()
    src = np.moveaxis(states, row_dim, 0)
    dst = np.moveaxis(got, row_dim, 0)
    for j, p in enumerate(parents):
        if p // beams != j // beams or p < 0:
            continue
        if lengths is None:
            dst[j] = src[p]
            continue
        d = (row_dim + 1 if length_dim is None else length_dim % states.ndim) - 1   # of a row, whose own dimension is gone
        n = min(max(int(lengths[p]), 0), src[p].shape[d])
        part = (slice(None),) * d + (slice(0, n),)
        dst[j][part] = src[p][part]
    return got
