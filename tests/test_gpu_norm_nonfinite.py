"""The norm's backward where dy, x or the statistics are not finite: an
element of dy that is 0 contributes 0 whatever lies beside it, and everything
else follows IEEE evaluation of the formula."""
import numpy as np
import pytest

import ops_reference as R
from gpu_common import dev, log

pytestmark = pytest.mark.gpu


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy()


def _grads(x, w, mean, rstd, dy, kind):
    """dx, dw, db in float64."""
    x, w, dy = (a.astype(np.float64) for a in (x, w, dy))
    r = rstd.astype(np.float64)[:, None]
    m = mean.astype(np.float64)[:, None] if kind == "layer" else 0.0
    with np.errstate(all="ignore"):
        xh = (x - m) * r
        xs, ws = np.where(dy == 0, 0.0, xh), np.where(dy == 0, 0.0, w)
        g = dy * ws
        c1 = (g * xs).mean(1, keepdims=True)
        c2 = g.mean(1, keepdims=True) if kind == "layer" else 0.0
        dx = np.where((dy == 0).all(1, keepdims=True), 0.0, r * ((g - c2) - xh * c1))
        return dx, (dy * xs).sum(0), dy.sum(0)


def _check(x, w, dy, kind, eps, what, y_t="f32"):
    import torch
    import cross_entropy_amd as lm
    t = {"f32": torch.float32, "bf16": torch.bfloat16}[y_t]
    xd, wd, dd = dev(x).to(t), dev(w), dev(dy).to(t)
    _, mean, rstd = lm.norm_forward(xd, wd, None, eps, kind)
    got = lm.norm_backward(xd, wd, mean, rstd, dd, kind, with_bias=True)
    torch.cuda.synchronize()
    x, dy, mean, rstd = (_np(a) for a in (xd, dd, mean, rstd))
    want = _grads(x, w, mean, rstd, dy, kind)
    # the bounds of the finite results: from the finite values (the others make every result they enter non-finite)
    fin = lambda a: None if a is None else np.where(np.isfinite(a), a, 0)   # noqa: E731
    bounds = R.norm_grad_bounds(fin(x), w, fin(mean), fin(rstd), fin(dy), kind, y_t, "f32")
    for a, b, e, n in zip(got, want, bounds, ("dx", "dw", "db")):
        R.check(_np(a), b, e, f"{what} {n}")
    return want


@pytest.mark.parametrize("N", [8, 600])   # the weight's gradient by columns and by partial sums
@pytest.mark.parametrize("H", [6, 40, 202, 520, 1000, 4100, 9000])
@pytest.mark.parametrize("y_t", ["f32", "bf16"])
def test_norm_of_a_gradient_that_is_not_finite(N, H, y_t):
    """NaN and infinities in dy reach dx and dweight where the weight is 0 and
    where x has its mean's value (0 times them is NaN)."""
    rng = np.random.default_rng(H)
    x = rng.standard_normal((N, H)).astype(np.float32)
    x[:4] = np.where(np.arange(H) % 2, 1.0, -1.0)     # their mean is exactly 0,
    x[:4, 2:4] = 0.0                                  # and their value there
    w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    w[1] = w[4] = 0.0
    dy = rng.standard_normal((N, H)).astype(np.float32)
    dy[0, 2] = np.nan      # xh = 0
    dy[1, 3] = np.inf      # xh = 0
    dy[2, 1] = np.nan      # weight 0
    dy[3, 4] = -np.inf     # weight 0
    dy[4, 5] = np.inf
    dy[5] = 0.0
    for kind in ("layer", "rms"):
        log(f"[norm] non-finite dy N={N} H={H} {kind} {y_t}")
        dx, dw, db = _check(x, w, dy, kind, 1e-6, f"N={N} H={H} {kind}", y_t)
        assert np.isnan(dx[[0, 1, 2, 3]]).any(1).all() and np.isnan(dx[[0, 2]]).all() and np.isnan(dw[[1, 2, 3]]).all()
        assert np.isfinite(dx[5:]).all() and (H == 6 or np.isfinite(dw[6:]).all())


@pytest.mark.parametrize("N", [8, 600])
@pytest.mark.parametrize("H", [6, 202, 1000, 4100, 9000])
def test_norm_of_rows_that_are_not_finite(N, H):
    """Under an incoming gradient of 0 a row of NaN, of infinities, or of
    zeros without an eps adds nothing; under any other it makes its results
    NaN. RMS: an infinity in x alone takes the row's scale to 0."""
    rng = np.random.default_rng(H + 1)
    x = rng.standard_normal((N, H)).astype(np.float32)
    w = (1 + 0.2 * rng.standard_normal(H)).astype(np.float32)
    dy = rng.standard_normal((N, H)).astype(np.float32)
    x[0], x[1], x[2, 3], x[3] = np.nan, np.inf, -np.inf, 0.0
    x[5, 2] = np.inf
    dy[:4] = 0.0
    dy[1] = -0.0
    for kind in ("layer", "rms"):
        log(f"[norm] non-finite rows N={N} H={H} {kind}")
        y = dy.copy()
        y[5] = 0.0
        dx, dw, db = _check(x, w, y, kind, 0.0, f"dead N={N} H={H} {kind}")
        assert (dx[:4] == 0).all() and np.isfinite(dx).all() and np.isfinite(dw).all()
        y[5], y[5, 2] = dy[5], 0.0                    # the infinity under a 0 of a gradient that is not 0
        dx, dw, db = _check(x, w, y, kind, 0.0, f"live N={N} H={H} {kind}")
        assert np.isnan(dx[5, 2]) and np.isfinite(np.delete(dx, 5, 0)).all()
        y[0] = dy[6]
        y[3, 1] = 1.0                                 # a row of zeros, its scale infinite
        dx, dw, db = _check(x, w, y, kind, 0.0, f"NaN N={N} H={H} {kind}")
        assert np.isnan(dx[[0, 3]]).all() and np.isfinite(dx[[1, 2, 4]]).all()
