"""The norm in front of the head (lmhead_logps_norm_fwd / _bwd) through the C
ABI and its front ends, against float64, within bounds derived from the
roundings (tests/ops_reference.py)."""
import numpy as np
import pytest

import ops_reference as R
from gpu_common import dev, log

pytestmark = pytest.mark.gpu


def _t(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _put(a, t):
    return None if a is None else dev(np.asarray(a, np.float32)).to(_t(t))


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy()


def _data(seed, N, H, x_t, w_t, y_t, weight=True, bias=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((N, H)) * np.exp(rng.standard_normal((N, 1))) + rng.standard_normal((1, H))
    x = _put(x, x_t)
    w = _put(1 + 0.2 * rng.standard_normal(H), w_t) if weight else None
    b = _put(0.3 * rng.standard_normal(H), w_t) if bias else None
    dy = rng.standard_normal((N, H))
    dy[rng.random(N) < 0.1] = 0.0
    return x, w, b, _put(dy, y_t)


def _check(x, w, b, dy, kind, eps=1e-6, y_t="bf16", g_t=None, what=""):
    import torch
    import cross_entropy_amd as lm
    xt = "f32" if x.dtype == torch.float32 else "bf16"
    y, mean, rstd = lm.norm_forward(x, w, b, eps, kind, _t(y_t))
    gd = None if g_t is None else _t(g_t)
    dx, dw, db = lm.norm_backward(x, w, mean, rstd, dy, kind, with_weight=True, with_bias=True, grad_dtype=gd)
    torch.cuda.synchronize()
    X, Wn, B, DY = _np(x), _np(w), _np(b), _np(dy)
    ry, rm, rr = R.norm(X, Wn, B, eps, kind)
    ey, em, er = R.norm_bounds(X, Wn, B, eps, kind, y_t)
    R.check(_np(y), ry, ey, what + " y")
    R.check(_np(rstd), rr, er, what + " rstd")
    if kind == "layer":
        R.check(_np(mean), rm, em, what + " mean")
    else:
        assert mean is None
    gt = "f32" if dw.dtype == torch.float32 else "bf16"
    st = (_np(mean), _np(rstd))
    for got, want, bound, n in zip((dx, dw, db), R.norm_grads(X, Wn, *st, DY, kind),
                                   R.norm_grad_bounds(X, Wn, *st, DY, kind, xt, gt), ("dx", "dw", "db")):
        R.check(_np(got), want, bound, f"{what} {n}")
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 63, 64, 65, 320, 511, 512, 513, 1001, 1536, 2048, 2559, 2560, 2561, 4096,
                               5000, 6143, 8192, 8200, 12289, 16383, 16384])
@pytest.mark.parametrize("N", [1, 3, 70, 513])
def test_norm_sizes(N, H):
    """Every row shape of the kernels and its edges, both kinds, in turn with
    the types; the weight's gradient by columns and (513 rows) by partial sums."""
    k = H + N
    x_t, y_t = (("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32"))[k % 3]
    w_t = ("bf16", "f32")[k // 3 % 2]
    for kind in ("layer", "rms"):
        log(f"[norm] N={N} H={H} {kind} x={x_t} y={y_t} w={w_t}")
        x, w, b, dy = _data(k, N, H, x_t, w_t, y_t)
        _check(x, w, b, dy, kind, y_t=y_t, what=f"N={N} H={H} {kind}")


@pytest.mark.parametrize("x_t,y_t", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("w_t", ["bf16", "f32", None])
@pytest.mark.parametrize("g_t", ["bf16", "f32"])
def test_norm_types(x_t, y_t, w_t, g_t):
    log(f"[norm] types x={x_t} y={y_t} w={w_t} gradients={g_t}")
    for kind in ("layer", "rms"):
        x, w, b, dy = _data(5, 1237, 600, x_t, w_t or "f32", y_t, weight=w_t is not None, bias=w_t is not None)
        _check(x, w, b, dy, kind, y_t=y_t, g_t=g_t, what=f"{kind} {x_t} {y_t} {w_t}")


@pytest.mark.parametrize("N,H", [(512, 33), (512, 2560), (4096, 256), (17000, 128), (5003, 2564)])
def test_norm_many_rows(N, H):
    """Threads that walk several rows."""
    log(f"[norm] N={N} H={H}")
    x, w, b, dy = _data(N, N, H, "bf16", "bf16", "bf16")
    _check(x, w, b, dy, "layer", g_t="f32", what=f"N={N} H={H}")


def test_norm_large_mean_and_small_variance():
    """Centred before squared: a mean a thousand times the spread costs the
    variance no digits but those that x itself has lost."""
    rng = np.random.default_rng(3)
    x = dev((1000.0 + rng.standard_normal((33, 777))).astype(np.float32))
    dy = dev(rng.standard_normal((33, 777)).astype(np.float32))
    _check(x, None, None, dy, "layer", y_t="f32", what="large mean")
    x = dev(np.full((5, 100), 3.25, np.float32))       # no variance: eps alone
    dy = dev(rng.standard_normal((5, 100)).astype(np.float32))
    _check(x, None, None, dy, "layer", eps=1e-5, y_t="f32", what="constant rows")
    x = dev(np.zeros((5, 100), np.float32))
    _check(x, None, None, dy, "rms", eps=1e-5, y_t="f32", what="zero rows")


def test_norm_masked_rows_do_not_spread():
    """Rows whose dy is 0 add nothing, whatever x and their statistics hold;
    other rows' outputs do not see them."""
    import torch
    import cross_entropy_amd as lm
    for N, H in ((90, 200), (90, 4096), (600, 200), (600, 4096)):
        x, w, b, dy = _data(7, N, H, "f32", "f32", "f32")
        bad = torch.tensor([0, 31, 32, 89], device="cuda")
        dy[bad] = 0.0
        y, mean, rstd = lm.norm_forward(x, w, b)
        ref = lm.norm_backward(x, w, mean, rstd, dy, with_bias=True)
        x2 = x.clone()
        x2[bad[0]] = float("nan")
        x2[bad[1]] = float("inf")
        x2[bad[2], 5] = float("-inf")
        x2[bad[3], 0] = float("nan")
        y2, mean2, rstd2 = lm.norm_forward(x2, w, b)
        got = lm.norm_backward(x2, w, mean2, rstd2, dy, with_bias=True)
        torch.cuda.synchronize()
        keep = torch.ones(N, dtype=torch.bool, device="cuda")
        keep[bad] = False
        assert torch.equal(y[keep], y2[keep])
        assert not torch.isfinite(y2[bad]).all(1).any()
        for a, c in zip(ref, got):
            assert torch.equal(a, c)
        assert (got[0][bad] == 0).all()


def test_norm_writes_only_its_rows():
    """Odd rows between others: nothing before or behind them is written."""
    import torch
    import cross_entropy_amd as lm
    for N, H, t in ((5, 1001, torch.bfloat16), (3, 7, torch.bfloat16), (4, 2563, torch.float32)):
        big = torch.full((N + 2, H), 3.0, device="cuda", dtype=t)
        gb = torch.full((N + 2, H), 5.0, device="cuda", dtype=t)
        x = torch.randn(N, H, device="cuda").to(t)
        st = torch.full((2, N + 2), 9.0, device="cuda")
        lm.lmhead_logps_norm_fwd(x, None, None, 1e-6, "layer", big[1:N + 1], st[0, 1:N + 1], st[1, 1:N + 1])
        w = torch.full((3, H), 4.0, device="cuda")
        lm.lmhead_logps_norm_bwd(x, None, "layer", st[0, 1:N + 1], st[1, 1:N + 1], big[1:N + 1], gb[1:N + 1], w[1], None,
                                 0, lm.norm_workspace_for(x))
        torch.cuda.synchronize()
        assert (big[0] == 3).all() and (big[-1] == 3).all() and (gb[0] == 5).all() and (gb[-1] == 5).all()
        assert (st[:, 0] == 9).all() and (st[:, -1] == 9).all() and (w[0] == 4).all() and (w[2] == 4).all()
        assert not (big[1:N + 1] == 3).all()


def test_norm_beyond_32_bit_offsets():
    """5.2 GB of rows: the last ones give the bits of a call of their own."""
    import torch
    import cross_entropy_amd as lm
    N, H = 640000, 4096
    x = torch.empty(N, H, device="cuda", dtype=torch.bfloat16)
    for r in range(0, N, 80000):
        x[r:r + 80000] = torch.randn(80000, H, device="cuda")
    y, mean, rstd = lm.norm_forward(x)
    dx, _, _ = lm.norm_backward(x, None, mean, rstd, y, with_weight=False)
    for rows in (slice(0, 50), slice(N - 50, N)):
        part = x[rows].contiguous()
        y2, m2, r2 = lm.norm_forward(part)
        d2, _, _ = lm.norm_backward(part, None, m2, r2, y2, with_weight=False)
        torch.cuda.synchronize()
        for a, b in ((y[rows], y2), (mean[rows], m2), (rstd[rows], r2), (dx[rows], d2)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("N", [501, 700])
def test_norm_adds_into_gradients(N):
    import torch
    import cross_entropy_amd as lm
    x, w, b, dy = _data(11, N, 384, "bf16", "bf16", "bf16")
    y, mean, rstd = lm.norm_forward(x, w, b)
    dx, dw, db = lm.norm_backward(x, w, mean, rstd, dy, with_bias=True, grad_dtype=torch.float32)
    for t in (torch.float32, torch.bfloat16):
        pw, pb = torch.randn(384, device="cuda").to(t), torch.randn(384, device="cuda").to(t)
        aw, ab = pw.clone(), pb.clone()
        lm.norm_backward(x, w, mean, rstd, dy, with_bias=True, dweight=aw, dbias=ab, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(aw, (pw.float() + dw).to(t)) and torch.equal(ab, (pb.float() + db).to(t))
    only = lm.norm_backward(x, w, mean, rstd, dy, with_weight=False, with_bias=True, grad_dtype=torch.float32)
    none = lm.norm_backward(x, w, mean, rstd, dy, with_weight=False)
    torch.cuda.synchronize()
    assert only[1] is None and torch.equal(only[2], db) and none[1:] == (None, None)
    assert torch.equal(only[0], dx) and torch.equal(none[0], dx)


def test_norm_without_rows():
    import torch
    import cross_entropy_amd as lm
    x = torch.empty(0, 96, device="cuda")
    y, mean, rstd = lm.norm_forward(x)
    dw = torch.full((96,), 7.0, device="cuda")
    db = torch.full((96,), 7.0, device="cuda", dtype=torch.bfloat16)
    lm.norm_backward(x, None, mean, rstd, x, with_bias=True, dweight=dw, dbias=dw.clone(), accumulate=True)
    assert (dw == 7).all()
    lm.norm_backward(x, None, mean, rstd, x, dweight=dw)
    lm.norm_backward(x, None, mean, rstd, x, with_weight=False, dbias=db)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


def test_norm_gradient_against_differences():
    """The autograd front end's gradients against central differences of the
    loss sum(y g) in float64. The third derivative's share at step 1e-4 is
    below 1e-8 of values of this size; the rest is the bound of the gradient."""
    import torch
    import cross_entropy_amd as lm
    rng = np.random.default_rng(2)
    N, H = 6, 40
    for kind in ("layer", "rms"):
        x, w, b, g = (rng.standard_normal(s).astype(np.float32) for s in ((N, H), (H,), (H,), (N, H)))
        leaves = [dev(a).requires_grad_() for a in (x, w, b)]
        y = lm.lmhead_norm(leaves[0].view(2, 3, H), leaves[1], leaves[2], 1e-3, kind)
        assert y.shape == (2, 3, H)
        (y.view(N, H) * dev(g)).sum().backward()
        f = lambda *a: (R.norm(*a, 1e-3, kind)[0] * g).sum()  # noqa: E731
        _, mean, rstd = R.norm(x, w, b, 1e-3, kind)
        bounds = R.norm_grad_bounds(x, w, mean, rstd, g, kind, "f32", "f32")
        # the front end's statistics are themselves rounded: their error as in the forward's bound, through every gradient
        _, em, er = R.norm_bounds(x, w, b, 1e-3, kind, "f32")
        rel = float((er / rstd).max() + (em * rstd).max())
        for i, (leaf, a) in enumerate(zip(leaves, (x, w, b))):
            d = rng.standard_normal(a.shape)
            h = 1e-4
            args = [t.astype(np.float64) for t in (x, w, b)]
            plus, minus = list(args), list(args)
            plus[i], minus[i] = args[i] + h * d, args[i] - h * d
            want = (f(*plus) - f(*minus)) / (2 * h)
            got = (_np(leaf.grad).astype(np.float64) * d).sum()
            size = np.abs(_np(leaf.grad) * d).sum() + (np.abs(g) * 8).sum() * (i == 0)
            lim = (np.broadcast_to(bounds[i], a.shape) * np.abs(d)).sum() + 8 * rel * size + 1e-6 * max(1.0, abs(want))
            assert abs(got - want) <= lim, (kind, i, got, want, lim)


def test_norm_refuses_what_it_does_not_take():
    import torch
    import cross_entropy_amd as lm
    x = torch.randn(4, 64, device="cuda")
    for bad, err in (((x.half(),), TypeError), ((x.t(),), ValueError), ((x, x[0].half()), TypeError),
                     ((x, x[0, :32]), ValueError), ((x, x[0], x[0].bfloat16()), TypeError)):
        with pytest.raises(err):
            lm.norm_forward(*bad)
    with pytest.raises(ValueError):
        lm.norm_forward(x, kind="group")
    with pytest.raises(lm.LmheadError):
        lm.norm_forward(x.bfloat16(), out_dtype=torch.float32)
    with pytest.raises(lm.LmheadError):
        lm.norm_forward(torch.randn(1, 16392, device="cuda"))
    y, mean, rstd = lm.norm_forward(x)
    with pytest.raises(ValueError):
        lm.norm_backward(x, None, mean, rstd, x[:2])
    with pytest.raises(ValueError):
        lm.norm_backward(x, None, mean[:3], rstd, x)
    with pytest.raises(ValueError):
        lm.norm_backward(x, None, mean, rstd, x, accumulate=True)
    with pytest.raises(ValueError):
        lm.norm_backward(x, None, mean, rstd, x.cpu())
