"""The norm and the distillation loss in float64 numpy, from their
definitions, and the error bounds that the GPU tests hold results to. Shares
no code with the library."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24                        # float32's largest relative rounding error
HALF = {"f32": U, "bf16": 2.0 ** -8}  # likewise per stored type
SUMS = 256                            # more additions than any float32 sum of the norm has in sequence


def norm(x, w, b, eps, kind):
    """y, mean, rstd of rows x [N, H]."""
    x = x.astype(np.float64)
    mean = x.mean(1) if kind == "layer" else np.zeros(len(x))
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if w is not None:
        y = y * w.astype(np.float64)
    if b is not None:
        y = y + b.astype(np.float64)
    return y, mean, rstd


def norm_bounds(x, w, b, eps, kind, y_type):
    """Largest errors of (y, mean, rstd)."""
    y, mean, rstd = norm(x, w, b, eps, kind)
    x = np.abs(x.astype(np.float64))
    e_mean = SUMS * U * x.mean(1) if kind == "layer" else np.zeros(len(x))
    # a mean off by e moves the variance by e^2; the sum of squares is SUMS roundings off, its root half of that
    e_rstd = rstd * (SUMS * U + 0.5 * (e_mean * rstd) ** 2)
    wa = np.ones(x.shape[1]) if w is None else np.abs(w.astype(np.float64))
    ba = np.zeros(x.shape[1]) if b is None else np.abs(b.astype(np.float64))
    scaled = np.abs(y) + ba
    e_y = scaled * (8 * U) + (scaled / rstd[:, None]) * e_rstd[:, None] + (rstd * e_mean)[:, None] * wa
    return e_y * (1 + HALF[y_type]) + HALF[y_type] * np.abs(y), e_mean, e_rstd


def norm_grads(x, w, mean, rstd, dy, kind):
    """dx, dw, db with the given statistics. A zero of dy contributes a zero."""
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    r = rstd.astype(np.float64)[:, None]
    m = mean.astype(np.float64)[:, None] if kind == "layer" else 0.0
    with np.errstate(all="ignore"):
        xh = (x - m) * r
        g = dy if w is None else np.where(dy == 0, 0.0, dy * w.astype(np.float64))
        gx = np.where(g == 0, 0.0, g * xh)
        c1 = gx.mean(1, keepdims=True)
        c2 = g.mean(1, keepdims=True) if kind == "layer" else np.zeros_like(c1)
        dead = ~np.any(dy != 0, axis=1, keepdims=True)
        dx = np.where(dead, 0.0, r * (g - c2 - xh * c1))
        dw = np.where(dy == 0, 0.0, dy * xh)
    return dx, dw.sum(0), dy.sum(0)


def norm_grad_bounds(x, w, mean, rstd, dy, kind, x_type, g_type):
    """Largest errors of (dx, dw, db)."""
    dx, dw, db = norm_grads(x, w, mean, rstd, dy, kind)
    x, dy = x.astype(np.float64), dy.astype(np.float64)
    r = np.abs(rstd.astype(np.float64))[:, None]
    m = mean.astype(np.float64)[:, None] if kind == "layer" else 0.0
    xh = np.abs(x - m) * r
    g = np.abs(dy if w is None else dy * w.astype(np.float64))
    c1, c2 = (g * xh).mean(1, keepdims=True), g.mean(1, keepdims=True)
    e_dx = r * U * ((SUMS + 8) * (c2 + xh * c1) + 8 * g)
    e_dx = e_dx * (1 + HALF[x_type]) + HALF[x_type] * np.abs(dx)
    e_dw = (SUMS + 4) * U * (np.abs(dy) * xh).sum(0) + HALF[g_type] * np.abs(dw)
    e_db = (SUMS + 4) * U * np.abs(dy).sum(0) + HALF[g_type] * np.abs(db)
    return e_dx, e_dw * (1 + HALF[g_type]), e_db * (1 + HALF[g_type])


def teacher_q(ids, t, tlse, V, T):
    """live, log q (0 where q = 0) and q of teacher entries [N, K]."""
    live = (ids >= 0) & (ids < V)
    with np.errstate(all="ignore"):
        t = np.where(live, t.astype(np.float64) / T, -np.inf)
        if tlse is not None:
            lq = t - tlse.astype(np.float64)[:, None]
        else:
            m = t.max(1, keepdims=True)
            m = np.where(np.isneginf(m), 0.0, m)
            lq = t - (m + np.log(np.exp(t - m).sum(1, keepdims=True)))
        none = np.isneginf(t)
        q = np.where(none, 0.0, np.exp(lq))
        lq = np.where(none, 0.0, lq)
    return live, lq, q


class Distill:
    """The loss, its statistics, its cotangent of the logits and its gradients,
    for hidden [N, H] and W [V, H] as float arrays."""

    def __init__(self, h, W, targets, ids, t, tlse, T):
        self.h, self.W, self.T, self.ids = h.astype(np.float64), W.astype(np.float64), T, ids
        V = W.shape[0]
        self.live, self.lq, self.q = teacher_q(ids, t, tlse, V, T)
        self.hard = np.zeros(len(h), bool) if targets is None else (targets >= 0) & (targets < V)
        self.targets = np.where(self.hard, 0 if targets is None else targets, 0)
        self.used = self.live.any(1) | self.hard
        hh = np.where(self.used[:, None], self.h, 0.0)   # a masked token's row is not looked at
        self.h = hh
        z = hh @ self.W.T / T
        m = z.max(1, keepdims=True)
        lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
        self.logs = z - lse[:, None]
        rows = np.arange(len(h))[:, None]
        self.top = np.where(self.live, self.logs[rows, np.where(self.live, ids, 0)], 0.0)
        self.kl = np.where(self.q > 0, self.q * (self.lq - self.top), 0.0).sum(1)
        self.kl = np.where(np.isnan(self.q).any(1), np.nan, self.kl)
        self.logp = np.where(self.hard, self.logs[rows[:, 0], self.targets], 0.0)
        self.lse = np.where(self.used, lse, 0.0)
        # a logit is H float32 products and sums off at most, and its division by T; a log-sum-exp as much as its logits,
        # its own sum (pairs of 32 to 128 terms, tiles and splits in sequence: below 2^10 additions) and its logarithm
        H = h.shape[1]
        mag = (np.abs(hh) @ np.abs(self.W).T).max(1) / T
        self.e_z = (H + 8) * U * mag
        self.e_lse = self.e_z + (2 ** 10 + 8) * U + 8 * U * (np.abs(lse) + mag)
        self.e_top = (self.e_z + self.e_lse)[:, None] + 4 * U * np.abs(self.top)
        Q = self.q.sum(1)
        with np.errstate(all="ignore"):
            tmag = np.where(self.q > 0, np.abs(np.where(self.live, t, 0).astype(np.float64) / T), 0.0)
        # log q: the division's rounding, the shift's and its sum's (K in sequence at most 16, then 6 levels)
        self.e_lq = 64 * U * (1.0 + tmag.max(1, initial=0.0) + np.abs(self.lq).max(1, initial=0.0))
        size = (self.q * (np.abs(self.lq) + np.abs(self.top))).sum(1)
        self.e_kl = Q * (self.e_z + self.e_lse + self.e_lq) + size * (64 * U + self.e_lq)
        self.e_logp = self.e_z + self.e_lse + 4 * U * np.abs(self.logp)

    def backward(self, g_kl, g_logp, grad_type):
        """dh, dW and their largest errors."""
        N, V = self.logs.shape
        gk = np.zeros(N) if g_kl is None else g_kl.astype(np.float64)
        gl = np.zeros(N) if g_logp is None else np.where(self.hard, g_logp.astype(np.float64), 0.0)
        gk = np.where(self.used, gk, 0.0)
        q = np.where((gk != 0)[:, None], self.q, 0.0)
        Q = q.sum(1)
        p = np.exp(self.logs) * self.used[:, None]
        qv = np.zeros((N, V))
        rows = np.broadcast_to(np.arange(N)[:, None], self.ids.shape)
        np.add.at(qv, (rows[self.live], self.ids[self.live]), q[self.live])
        one = np.zeros((N, V))
        one[np.arange(N)[self.hard], self.targets[self.hard]] = 1.0
        dz = (gk[:, None] * (Q[:, None] * p - qv) + gl[:, None] * (one - p)) / self.T
        # each entry of dz: p off by the exponent's error, q by log q's, then one rounding to bf16
        e_p = 2 * (self.e_z + self.e_lse) + 16 * U
        e = ((np.abs(gk) * Q + np.abs(gl)) * (e_p + self.e_lq + 16 * U))[:, None] * p
        e = (e + np.abs(gk)[:, None] * qv * (self.e_lq + 16 * U)[:, None] + np.abs(gl)[:, None] * one * 4 * U) / self.T
        e = e * (1 + HALF["bf16"]) + HALF["bf16"] * np.abs(dz) + 2.0 ** -133   # bf16's half step at its smallest
        dh, dW = dz @ self.W, dz.T @ self.h
        # the products' float32 sums: at most V (or N) terms in sequence
        a_h, a_W = np.abs(dz) @ np.abs(self.W), np.abs(dz).T @ np.abs(self.h)
        half = HALF[grad_type]
        e_h = (e @ np.abs(self.W) + V * U * a_h) * (1 + half) + half * np.abs(dh)
        e_W = (e.T @ np.abs(self.h) + N * U * a_W) * (1 + half) + half * np.abs(dW)
        e_h = np.where(self.used[:, None], e_h, 0.0)
        return dh, dW, e_h, e_W


def check(got, want, bound, what):
    """|got - want| <= bound everywhere; NaN and infinities in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: other infinities"
    err = np.abs(got - want)[fine]
    lim = np.broadcast_to(bound, want.shape)[fine]
    bad = ~(err <= lim)
    if bad.any():
        k = int(np.argmax(np.where(bad, err / np.maximum(lim, 1e-300), 0)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.size} outside; worst {got[fine][k]!r} for "
                             f"{want[fine][k]!r}, {err[k]:.3e} off where {lim[k]:.3e} is allowed")
