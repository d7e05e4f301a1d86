"""The distillation head (lmhead_logps_distill_fwd / _bwd) through the C ABI
and its front end, against float64, within bounds derived from the roundings
(tests/ops_reference.py); and the norm, the head and the loss together."""
import numpy as np
import pytest

import ops_reference as R
from gpu_common import dev, dev_bits, log
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _case(seed, N, H, V, K, T=1.0, t_type="f32", tail=False, hard=True, pad=0.1, lean=True):
    """Arrays of one case: bf16 patterns of hidden and W, targets (or None),
    ids, teacher (float32 values of its type), teacher_lse (or None)."""
    rng = np.random.default_rng(seed)
    W = f32_to_bf16_bits((0.1 * rng.standard_normal((V, H))).astype(np.float32))
    ids = rng.integers(0, V, (N, K)).astype(np.int32)
    h = rng.standard_normal((N, H))
    if lean:                                   # the student puts weight on the first ids
        Wf = bf16_bits_to_f32(W)
        h += 4.0 / (0.01 * H) * Wf[ids[:, 0]]
        if K > 1:
            h += 2.0 / (0.01 * H) * Wf[ids[:, 1]]
    h = f32_to_bf16_bits(h.astype(np.float32))
    t = 8.0 - 1.3 * np.log1p(np.arange(K)) + rng.standard_normal((N, K))
    t = t.astype(np.float32)
    if K > 1:
        t[rng.random((N, K)) < 0.03] = -np.inf
        t[:, 0] = 8.0
    if t_type == "bf16":
        t = bf16_bits_to_f32(f32_to_bf16_bits(t))
    targets = None
    if hard:
        targets = rng.integers(0, V, N).astype(np.int32)
        same = rng.random(N) < 0.5
        targets[same] = ids[same, rng.integers(0, K)]
        targets[rng.random(N) < 0.1] = -1
    if K > 1:                                  # shorter lists
        short = rng.random(N) < 0.3
        cut = rng.integers(1, K + 1, N)
        ids[short[:, None] & (np.arange(K)[None] >= cut[:, None])] = -1
    n_pad = int(pad * N)
    if n_pad:
        ids[N - n_pad:] = -1
        if targets is not None:
            targets[N - n_pad:] = -1
    tlse = None
    if tail:
        with np.errstate(all="ignore"):
            m = np.where(np.isneginf(t), -np.inf, t / T)
            tlse = (np.log(np.exp(m - 10).sum(1)) + 10 + 0.3 * rng.random(N)).astype(np.float32)
    return h, W, targets, ids, t, tlse


def _put(h, W, targets, ids, t, tlse, t_type="f32"):
    import torch
    td = dev(t)
    return (dev_bits(h), dev_bits(W), None if targets is None else dev(targets), dev(ids),
            td.to(torch.bfloat16) if t_type == "bf16" else td, None if tlse is None else dev(tlse))


def _g(seed, N, hard):
    rng = np.random.default_rng(seed)
    return rng.standard_normal(N).astype(np.float32), (rng.standard_normal(N).astype(np.float32) if hard else None)


def _np(t):
    return None if t is None else t.detach().float().cpu().numpy()


def _forward_check(args, put, T, C, what):
    import torch
    import cross_entropy_amd as lm
    h, W, targets, ids, t, tlse = args
    hd, Wd, tg, idd, td, tl = put
    kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, C, tl, temperature=T)
    torch.cuda.synchronize()
    ref = R.Distill(bf16_bits_to_f32(h), bf16_bits_to_f32(W), targets, ids, t, tlse, T)
    R.check(_np(kl), ref.kl, ref.e_kl, what + " kl")
    R.check(_np(lse), ref.lse, np.where(ref.used, ref.e_lse, 0), what + " lse")
    R.check(_np(top), ref.top, np.where(ref.live, ref.e_top, 0), what + " logp_top")
    if targets is not None:
        R.check(_np(logp), ref.logp, np.where(ref.hard, ref.e_logp, 0), what + " logp")
    else:
        assert logp is None
    return ref, (kl, logp, lse, top)


def _check(args, T=1.0, C=64, t_type="f32", grads=("f32", "bf16"), what=""):
    import torch
    import cross_entropy_amd as lm
    put = _put(*args, t_type)
    ref, (kl, logp, lse, top) = _forward_check(args, put, T, C, what)
    hd, Wd, tg, idd, td, tl = put
    g_kl, g_logp = _g(1, len(args[0]), args[2] is not None)
    gk, gl = dev(g_kl), None if g_logp is None else dev(g_logp)
    for t in grads:
        dh, dW = lm.distill_backward(hd, Wd, tg, idd, td, C, logp, lse, top, gk, gl, tl, temperature=T,
                                     grad_dtype=torch.float32 if t == "f32" else torch.bfloat16)
        torch.cuda.synchronize()
        rh, rW, eh, eW = ref.backward(g_kl, g_logp, t)
        R.check(_np(dh), rh, eh, f"{what} dh {t}")
        R.check(_np(dW), rW, eW, f"{what} dW {t}")
    return ref


CASES = [
    # N, H, V, K, chunk, T, teacher, teacher_lse, hard
    (1, 64, 5, 1, 1, 1.0, "f32", False, True),
    (1, 128, 777, 3, 16, 1.0, "bf16", True, False),
    (5, 64, 1100, 1024, 8, 1.0, "f32", False, True),
    (17, 192, 300, 9, 64, 0.7, "bf16", False, True),
    (256, 256, 4096, 8, 128, 1.0, "f32", False, True),
    (300, 128, 1000, 16, 64, 2.0, "f32", True, True),
    (513, 256, 4097, 33, 4096, 1.0, "bf16", True, True),
    (700, 320, 3001, 64, 7, 1.0, "f32", True, False),     # a chunk_size below every block
    (2100, 128, 777, 17, 64, 1.0, "bf16", False, True),   # N > V: token blocks outer
    (70, 128, 20011, 12, 30, 1.0, "f32", True, True),     # split dh products, a ragged last
    (300, 192, 9000, 5, 4096, 2.0, "bf16", False, True),  # split over two token tiles in one block
    (1, 64, 40000, 1, 1, 1.0, "f32", False, True),
    (33, 320, 2000, 7, 64, 1.0, "bf16", False, True),     # few tokens at each count of their tiles
    (64, 64, 17, 5, 4096, 0.7, "f32", True, True),
    (65, 192, 5003, 9, 64, 1.0, "f32", False, True),
    (128, 448, 3000, 20, 64, 1.0, "bf16", True, False),
    (129, 128, 12345, 6, 4096, 2.0, "f32", False, True),
    (200, 512, 8000, 32, 128, 1.0, "f32", True, True),
    (256, 64, 1025, 3, 128, 1.0, "bf16", False, True),
    (257, 64, 1025, 3, 512, 1.0, "bf16", False, True),
    (128, 128, 24576, 6, 64, 1.0, "bf16", True, True),    # more tokens of a smaller vocabulary, at its limit and past it
    (128, 128, 24577, 6, 64, 1.0, "f32", False, True),
    (100, 576, 20000, 9, 64, 0.7, "f32", True, True),
    (192, 64, 16384, 6, 96, 1.0, "f32", False, True),
    (150, 320, 16385, 6, 512, 1.0, "bf16", True, False),
    (256, 192, 12288, 6, 128, 1.0, "f32", True, True),
    (250, 64, 12289, 6, 128, 2.0, "bf16", False, True),
    (40, 128, 3000, 6, 31, 1.0, "f32", False, True),      # a chunk_size below the tokens
    (3000, 128, 600, 4, 600, 1.0, "f32", False, True),    # split dW products
    (3000, 192, 9000, 5, 200, 1.0, "bf16", True, True),   # both split
    (1100, 64, 2500, 3, 64, 2.0, "f32", False, True),
    (130, 64, 70, 100, 32, 1.0, "f32", False, True),      # more entries than the vocabulary has ids
]


@pytest.mark.parametrize("N,H,V,K,C,T,t_type,tail,hard", CASES)
def test_distill(N, H, V, K, C, T, t_type, tail, hard):
    what = f"N={N} H={H} V={V} K={K} C={C} T={T} {t_type} tail={tail} hard={hard}"
    log(f"[distill] {what}")
    _check(_case(N + V + K, N, H, V, K, T, t_type, tail, hard), T, C, t_type, what=what)


@pytest.mark.parametrize("N,H,V,K,C,T,t_type,tail,hard", [
    (500, 64, 140001, 5, 7, 1.0, "f32", True, True),       # three vocabulary blocks, split dh products, a ragged last
    (2500, 64, 15001, 4, 64, 2.0, "bf16", False, True),    # two, dW products split too
    (15000, 64, 2500, 3, 64, 1.0, "f32", False, False),    # N > V: two token blocks, both split
    (12000, 64, 8001, 2, 1000, 1.0, "f32", True, True),    # two blocks each way
    (4000, 1536, 9000, 6, 64, 1.0, "bf16", True, True),    # two vocabulary blocks, nothing split
    (9000, 1536, 4000, 6, 64, 1.0, "f32", False, True),    # two token blocks, nothing split
])
def test_distill_several_blocks(N, H, V, K, C, T, t_type, tail, hard):
    what = f"blocks N={N} H={H} V={V} K={K} C={C} T={T} {t_type} tail={tail} hard={hard}"
    log(f"[distill] {what}")
    _check(_case(N + V + K, N, H, V, K, T, t_type, tail, hard), T, C, t_type, what=what)


def test_distill_random_shapes():
    rng = np.random.default_rng(77)
    for i in range(8):
        N, H, V = int(rng.integers(1, 900)), 64 * int(rng.integers(1, 6)), int(rng.integers(2, 2500))
        K, C, T = int(rng.integers(1, 140)), int(rng.integers(1, 600)), (1.0, 0.7, 3.0)[i % 3]
        t_type, tail, hard = ("f32", "bf16")[i % 2], i % 4 < 2, i % 3 != 0
        what = f"random {i}: N={N} H={H} V={V} K={K} C={C} T={T} {t_type} tail={tail} hard={hard}"
        log(f"[distill] {what}")
        _check(_case(500 + i, N, H, V, K, T, t_type, tail, hard, pad=0.2), T, C, t_type, what=what)


def test_distill_same_id_twice():
    """An id that the teacher lists several times: its q add up."""
    args = _case(8, 60, 128, 500, 12, hard=True, pad=0.0)
    h, W, targets, ids, t, tlse = args
    ids[:20, 5] = ids[:20, 2]
    ids[20:30] = ids[20:30, :1]            # one id in every place
    ids[30:40, 1] = ids[30:40, 0]
    targets[30:40] = ids[30:40, 0]
    ids[40:50, ::2] = ids[40:50, :1]
    _check(args, what="repeated ids")


def test_distill_student_equals_teacher():
    """Teacher logits that are the student's own: kl and its gradient vanish
    up to the roundings (Q p - q is formed before any rounding to bf16)."""
    import torch
    import cross_entropy_amd as lm
    N, H, V = 40, 64, 90
    h, W, _, _, _, _ = _case(9, N, H, V, 4, hard=False, pad=0.0)
    z = bf16_bits_to_f32(h).astype(np.float64) @ bf16_bits_to_f32(W).astype(np.float64).T
    ids = np.tile(np.arange(V, dtype=np.int32), (N, 1))
    args = (h, W, None, ids, z.astype(np.float32), None)
    ref = _check(args, what="student = teacher")
    # q and p each know their own log to e_lq and e_z + e_lse: the gradient is no larger than that
    hd, Wd, _, idd, td, _ = _put(*args)
    kl, _, lse, top = lm.distill_forward(hd, Wd, None, idd, td, 64)
    dh, _ = lm.distill_backward(hd, Wd, None, idd, td, 64, None, lse, top, torch.ones(N, device="cuda"))
    lim = (2 * (ref.e_z + ref.e_lse + ref.e_lq) + 64 * R.U)[:, None] * (np.exp(ref.logs) @ np.abs(ref.W)) * 2
    R.check(_np(dh), np.zeros((N, H)), lim, "vanishing dh")


def test_distill_masked_places_hold_anything():
    """NaN and infinities where nothing may look: the teacher logits of
    missing entries, masked tokens' hidden rows and teacher_lse, the rows of
    tokens without a cotangent."""
    import torch
    import cross_entropy_amd as lm
    args = _case(10, 120, 128, 700, 10, tail=True, hard=True, pad=0.1)
    h, W, targets, ids, t, tlse = args
    put = _put(*args)
    g_kl, g_logp = _g(2, 120, True)
    g_kl[:10] = 0.0

    def run(put, gk, gl):
        hd, Wd, tg, idd, td, tl = put
        kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
        out = lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, dev(gk), dev(gl), tl)
        torch.cuda.synchronize()
        return (kl, logp, lse, top) + out

    good = run(put, g_kl, g_logp)
    h2, t2, l2 = h.copy(), t.copy(), tlse.copy()
    dead = ids < 0
    t2[dead] = np.resize(np.float32([np.nan, np.inf, -np.inf, 3e38]), dead.sum())
    h2[108:] = 0x7FC0
    h2[109, 3] = 0x7F80
    l2[108:] = np.nan
    t2[:5] = np.nan                          # under g_kl = 0
    gk2, gl2 = g_kl.copy(), g_logp.copy()
    gk2[108:] = np.nan                       # masked tokens' cotangents
    gl2[108:] = np.inf
    bad = run(_put(h2, W, targets, ids, t2, l2), gk2, gl2)
    for i, (a, b, n) in enumerate(zip(good, bad, ("kl", "logp", "lse", "logp_top", "dh", "dW"))):
        if n == "kl":
            live = (ids[:5] >= 0).any(1)
            assert torch.isnan(b[:5][dev(live)]).all()
            a, b = a[5:], b[5:]
        assert torch.equal(a, b), n
    assert (good[0][108:] == 0).all() and (good[2][108:] == 0).all() and (good[4][108:] == 0).all()


def test_distill_empty_rows_with_any_cotangent():
    """A token without a teacher entry but with a hard target: its kl cotangent
    is not looked at. One with entries of no mass: kl 0, no gradient of it."""
    import torch
    import cross_entropy_amd as lm
    for N, V in ((20, 300), (300, 2000)):
        args = _case(30, N, 128, V, 6, hard=True, pad=0.0)
        h, W, targets, ids, t, tlse = args
        ids[:10] = -1
        targets[:10] = np.arange(10)
        t[10:15] = -np.inf
        hd, Wd, tg, idd, td, tl = _put(*args)
        g_kl, g_logp = _g(31, N, True)
        kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
        good = lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, dev(g_kl), dev(g_logp), tl)
        g_kl[:5], g_kl[5:10] = np.nan, np.inf
        bad = lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, dev(g_kl), dev(g_logp), tl)
        torch.cuda.synchronize()
        assert (kl[:15] == 0).all() and all(torch.equal(a, b) for a, b in zip(good, bad))
        ref = R.Distill(bf16_bits_to_f32(h), bf16_bits_to_f32(W), targets, ids, t, tlse, 1.0)
        g_kl[:10] = 0.0
        rh, rW, eh, eW = ref.backward(g_kl, g_logp, "f32")
        R.check(_np(good[0]), rh, eh, "dh")
        R.check(_np(good[1]), rW, eW, "dW")


def test_calls_on_a_stream_of_their_own():
    """The allocating helpers given a stream: results, workspaces and outputs
    belong to it, with work of the current stream around the call."""
    import torch
    import cross_entropy_amd as lm
    hd, Wd, tg, idd, td, tl = _put(*_case(32, 300, 128, 1300, 8, hard=True))
    gk, gl = (dev(a) for a in _g(8, 300, True))
    x = torch.randn(400, 640, device="cuda")

    def run(stream):
        kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl, stream=stream)
        out = (kl, logp, lse, top) + lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, gk, gl, tl,
                                                         stream=stream)
        y, mean, rstd = lm.norm_forward(x, stream=stream)
        return out + (y, mean, rstd) + lm.norm_backward(x, None, mean, rstd, y, with_bias=True, stream=stream)

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(8)]
        del junk
        got = run(stream)
        junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_distill_table_beyond_32_bit_offsets():
    """W and dW of 5.2 GB, ids at their end, for few tokens and for the tiles:
    against float32 on the rows that matter."""
    import torch
    import cross_entropy_amd as lm
    H, V, K = 4096, 640000, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    W = torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    for r in range(0, V, 80000):
        W[r:r + 80000] = 0.02 * torch.randn(80000, H, device="cuda", generator=gen)
    for N in (5, 300):
        log(f"[distill] beyond 32-bit offsets N={N}")
        h = torch.randn(N, H, device="cuda", generator=gen).bfloat16()
        ids = (V - 1 - torch.arange(N * K, device="cuda", dtype=torch.int32) * 7).view(N, K)
        t = torch.randn(N, K, device="cuda", generator=gen)
        tg = ids[:, 1].contiguous()
        kl, logp, lse, top = lm.distill_forward(h, W, tg, ids, t, 64)
        one = torch.ones(N, device="cuda")
        dh, dW = lm.distill_backward(h, W, tg, ids, t, 64, logp, lse, top, one, one, grad_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        z = torch.cat([h.float() @ W[r:r + 80000].float().t() for r in range(0, V, 80000)], 1)
        want = torch.logsumexp(z, 1)
        # either side's logits are 2^-24 (4096 + 8) sum |h w| off at most, sum |h w| = 4096 * 0.8 * 0.016 = 52 on average
        # and below 70; their log-sum-exps 2^-10 more (2^10 additions, logarithm, size 13)
        tol = 2 * 2.0 ** -24 * 4104 * 70 + 2 * 2.0 ** -10
        assert (lse - want).abs().max() <= tol
        assert (top - (z.gather(1, ids.long()) - want[:, None])).abs().max() <= 2 * tol
        q = torch.softmax(t, 1)
        p = torch.exp(z - want[:, None])
        dz = p * 0.0                             # Q = 1: g_kl Q - g_logp = 0 away from the special entries
        dz.scatter_add_(1, ids.long(), -q)
        dz.scatter_add_(1, tg.long()[:, None], one[:, None])
        last = slice(V - 8 * N * K, V)
        ref = dz[:, last].t() @ h.float()
        # each entry: q off by 2^-20, one rounding of the cotangent, float32 sums, the stored rounding
        lim = (2 * 2.0 ** -8 + 2.0 ** -12) * (dz[:, last].abs().t() @ h.float().abs()) + 1e-6
        assert ((dW[last].float() - ref).abs() <= lim).all()
        assert (dW[:V // 2].float().abs() <= 1e-5).all()
        rows = W[ids.long()].float()                                # [N, K, H]
        coef = dz.gather(1, ids.long())
        ref = (coef[:, :, None] * rows).sum(1)
        lim = (2 * 2.0 ** -8 + 2.0 ** -12) * (coef.abs()[:, :, None] * rows.abs()).sum(1) + 1e-5
        assert ((dh.float() - ref).abs() <= lim).all()
        del z, p, dz, dW


def test_distill_extreme_teacher_logits():
    """Lowest values, -inf rows, huge spreads; NaN and +inf stay in their row."""
    args = _case(11, 64, 64, 300, 6, hard=True, pad=0.0)
    h, W, targets, ids, t, tlse = args
    ids[:] = np.where(ids < 0, 7, ids)
    low = np.float32(-3.3895314e38)          # bfloat16's lowest
    t[0] = -np.inf
    t[1] = low
    t[2] = [low, low, 1.0, low, 2.0, -np.inf]
    t[3] = [300.0, -300.0, 0.0, 1e30, -1e30, 5.0]
    t[4] = 1e38
    for T, t_type in ((1.0, "f32"), (0.5, "bf16"), (4.0, "bf16")):
        tt = bf16_bits_to_f32(f32_to_bf16_bits(t)) if t_type == "bf16" else t.copy()
        if T == 0.5:
            tt[1] = -np.inf                  # low / 0.5 is beyond float32: as -inf
            tt[2, [0, 1, 3]] = -np.inf
            tt[4] = 1e37
        _check((h, W, targets, ids, tt, tlse), T, 64, t_type, what=f"extreme T={T}")
    t[5, 2] = np.nan
    t[6, 1] = np.inf
    put = _put(h, W, targets, ids, t, tlse)
    ref, out = _forward_check((h, W, targets, ids, t, tlse), put, 1.0, 64, "NaN rows")
    assert np.isnan(ref.kl[5:7]).all() and np.isfinite(ref.kl[7:]).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", [(330, 900), (330, 12000), (2000, 700), (500, 70001), (15000, 2500)])   # split dh, dW products; two blocks
def test_distill_adds_into_gradients(t, N, V):
    import torch
    import cross_entropy_amd as lm
    args = _case(12, N, 128, V, 7, hard=True)
    hd, Wd, tg, idd, td, tl = _put(*args)
    ty = torch.float32 if t == "f32" else torch.bfloat16
    g_kl, g_logp = _g(3, N, True)
    kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
    given = (hd, Wd, tg, idd, td, 64, logp, lse, top, dev(g_kl), dev(g_logp), tl)
    dh0, dW0 = lm.distill_backward(*given)
    ph, pW = torch.randn(N, 128, device="cuda").to(ty), torch.randn(V, 128, device="cuda").to(ty)
    dh, dW = ph.clone(), pW.clone()
    lm.distill_backward(*given, dh=dh, dW=dW, accumulate=True)
    torch.cuda.synchronize()
    masked = dev(~R.Distill(bf16_bits_to_f32(args[0]), bf16_bits_to_f32(args[1]), *args[2:], 1.0).used)
    assert masked.any() and torch.equal(dh[masked], ph[masked])
    # each sum of at most 16 blocks in float32, then the stored rounding
    for got, prev, g in ((dh, ph, dh0), (dW, pW, dW0)):
        want = _np(prev).astype(np.float64) + _np(g)
        size = np.abs(_np(prev)) + np.abs(_np(g))
        big = np.abs(want) * R.HALF[t] + 64 * R.U * (size + float(g.abs().max()))
        R.check(_np(got), want, big, "accumulated")


def test_distill_without_tokens():
    import torch
    import cross_entropy_amd as lm
    h = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(100, 64, device="cuda").bfloat16()
    ids = torch.empty(0, 3, device="cuda", dtype=torch.int32)
    t = torch.empty(0, 3, device="cuda")
    kl, logp, lse, top = lm.distill_forward(h, W, None, ids, t, 8)
    assert kl.shape == (0,) and top.shape == (0, 3)
    for ty in (torch.float32, torch.bfloat16):
        dW = torch.full((100, 64), 3.0, device="cuda", dtype=ty)
        dh = torch.empty(0, 64, device="cuda", dtype=ty)
        lm.distill_backward(h, W, None, ids, t, 8, None, lse, top, kl, dh=dh, dW=dW)
        torch.cuda.synchronize()
        assert (dW == 0).all()


def test_distill_is_the_head_without_its_loss():
    """Without a kl cotangent the backward is the head's own, and lse and logp
    are the head's within their bounds."""
    import torch
    import cross_entropy_amd as lm
    args = _case(13, 400, 128, 1500, 5, hard=True)
    hd, Wd, tg, idd, td, tl = _put(*args)
    kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
    hp, _, hl = lm.forward(hd, Wd, tg, 64)
    ref = R.Distill(bf16_bits_to_f32(args[0]), bf16_bits_to_f32(args[1]), *args[2:], 1.0)
    R.check(_np(logp), _np(hp), 2 * ref.e_logp, "logp")
    g = dev(_g(4, 400, True)[1])
    dh, dW = lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, None, g, tl)
    # the head's own backward on the same lse: targets' entries are formed the same way up to float32 roundings that
    # the rounding to bf16 may take to its other side
    h0, W0 = lm.backward(hd, Wd, tg, 64, lse, None, g)
    torch.cuda.synchronize()
    _, _, eh, eW = ref.backward(None, _np(g), "f32")
    R.check(_np(dh), _np(h0), 2 * eh, "dh")
    R.check(_np(dW), _np(W0), 2 * eW, "dW")


def test_distill_runs_repeat_bit_for_bit():
    import torch
    import cross_entropy_amd as lm
    args = _case(14, 600, 192, 2000, 40, tail=True, hard=True)
    hd, Wd, tg, idd, td, tl = _put(*args)
    gk, gl = (dev(a) for a in _g(5, 600, True))
    first = None
    for _ in range(3):
        kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 32, tl)
        out = (kl, logp, lse, top) + lm.distill_backward(hd, Wd, tg, idd, td, 32, logp, lse, top, gk, gl, tl,
                                                         grad_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_distill_gradient_against_differences():
    """The front end's gradients along random directions against central
    differences of the float64 loss, within the gradient's own bounds."""
    import torch
    import cross_entropy_amd as lm
    T, N, H, V, K = 1.5, 24, 64, 130, 6
    args = _case(15, N, H, V, K, T, tail=True, hard=True)
    h, W, targets, ids, t, tlse = args
    hd, Wd, tg, idd, td, tl = _put(*args)
    hd, Wd = (x.view(torch.bfloat16).clone().requires_grad_() for x in (hd, Wd))
    g_kl, g_logp = _g(6, N, True)
    kl, logp = lm.lmhead_distill(hd, Wd, idd, td, 16, tg, tl, T)
    ((kl * dev(g_kl)).sum() + (logp * dev(g_logp)).sum()).backward()
    hf, Wf = bf16_bits_to_f32(h).astype(np.float64), bf16_bits_to_f32(W).astype(np.float64)
    ref = R.Distill(hf, Wf, targets, ids, t, tlse, T)
    _, _, eh, eW = ref.backward(g_kl, g_logp, "bf16")

    def loss(a, b):
        r = R.Distill(a, b, targets, ids, t, tlse, T)
        return (r.kl * g_kl).sum() + (r.logp * g_logp).sum()

    rng = np.random.default_rng(0)
    for which, leaf, bound in ((0, hd, eh), (1, Wd, eW)):
        d = rng.standard_normal(leaf.shape)
        s = 1e-5
        step = (hf + s * d, hf - s * d) if which == 0 else (Wf + s * d, Wf - s * d)
        want = (loss(step[0], Wf) - loss(step[1], Wf) if which == 0 else loss(hf, step[0]) - loss(hf, step[1])) / (2 * s)
        got = (_np(leaf.grad).astype(np.float64) * d).sum()
        lim = (bound * np.abs(d)).sum() + 1e-5 * max(1.0, abs(want))
        assert abs(got - want) <= lim, (which, got, want, lim)


def _chain(lm, torch, x, w, b, Wd, idd, td, tg, kind, T):
    xs, ws, bs, Ws = (a.detach().clone().requires_grad_() for a in (x, w, b, Wd))
    kl, logp = lm.lmhead_distill(xs, Ws, idd, td, 64, tg, temperature=T, norm=lm.Norm(ws, bs, 1e-5, kind))
    (T * T * kl.sum() - 0.3 * logp.sum()).backward()
    return kl, logp, xs.grad, ws.grad, bs.grad, Ws.grad


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_head_and_distillation_together(kind):
    """A training step's end: stream -> norm -> head -> loss and back. The
    front end with norm= gives what the calls one by one give, bit for bit;
    each of those is held to float64 at its own inputs."""
    import torch
    import cross_entropy_amd as lm
    N, H, V, K, T = 200, 192, 1100, 12, 2.0
    h, W, targets, ids, t, tlse = _case(16, N, H, V, K, T, hard=True)
    rng = np.random.default_rng(1)
    x = dev((3.0 * bf16_bits_to_f32(h) + 0.5).astype(np.float32))
    x[N - 1] = float("nan")                      # a padded token's stream
    w, b = (dev((1.0 * i + 0.1 * rng.standard_normal(H)).astype(np.float32)) for i in (1, 0))
    Wd, tg, idd, td = dev_bits(W).view(torch.bfloat16), dev(targets), dev(ids), dev(t)
    kl, logp, gx, gw, gb, gW = _chain(lm, torch, x, w, b, Wd, idd, td, tg, kind, T)
    y, mean, rstd = lm.norm_forward(x, w, b, 1e-5, kind, torch.bfloat16)
    kl2, logp2, lse, top = lm.distill_forward(y, Wd, tg, idd, td, 64, temperature=T)
    gk, gl = torch.full((N,), T * T, device="cuda"), torch.full((N,), -0.3, device="cuda")
    dh, dW = lm.distill_backward(y, Wd, tg, idd, td, 64, logp2, lse, top, gk, gl, temperature=T,
                                 grad_dtype=torch.bfloat16)
    dx, dw, db = lm.norm_backward(x, w, mean, rstd, dh, kind, with_bias=True)
    torch.cuda.synchronize()
    for a, c, n in ((kl, kl2, "kl"), (logp, logp2, "logp"), (gx, dx, "dx"), (gw, dw, "dw"), (gb, db, "db"), (gW, dW, "dW")):
        assert torch.equal(a.detach(), c), n
    assert all(torch.isfinite(a).all() for a in (gx, gw, gb, gW)) and (gx[N - 1] == 0).all()
    ok = slice(0, N - 1)
    ry, _, _ = R.norm(_np(x)[ok], _np(w), _np(b), 1e-5, kind)
    ey, _, _ = R.norm_bounds(_np(x)[ok], _np(w), _np(b), 1e-5, kind, "bf16")
    R.check(_np(y)[ok], ry, ey, "y")
    yn = np.nan_to_num(_np(y))
    ref = R.Distill(yn, bf16_bits_to_f32(W), targets, ids, t, None, T)
    R.check(_np(kl2), ref.kl, ref.e_kl, "kl")
    rh, rW, eh, eW = ref.backward(_np(gk), _np(gl), "bf16")
    R.check(_np(dh), rh, eh, "dh")
    R.check(_np(dW), rW, eW, "dW")
    st = (None if mean is None else _np(mean)[ok], _np(rstd)[ok])
    bounds = R.norm_grad_bounds(_np(x)[ok], _np(w), *st, _np(dh)[ok], kind, "f32", "f32")
    for got, want, e, n in zip((_np(dx)[ok], _np(dw), _np(db)),
                               R.norm_grads(_np(x)[ok], _np(w), *st, _np(dh)[ok], kind), bounds, ("dx", "dw", "db")):
        R.check(got, want, e, n)


def test_head_front_end_with_norm():
    """lmhead_logps with norm= is the norm followed by the head."""
    import torch
    import cross_entropy_amd as lm
    N, H, V = 130, 128, 600
    h, W, targets, _, _, _ = _case(17, N, H, V, 3)
    x = dev_bits(h).view(torch.bfloat16)
    Wd, tg = dev_bits(W).view(torch.bfloat16), dev(targets)
    w = torch.rand(H, device="cuda").bfloat16() + 0.5
    a = [t.detach().clone().requires_grad_() for t in (x, w, Wd)]
    logp, ent = lm.lmhead_logps(a[0], a[2], tg, 64, norm=lm.Norm(a[1], kind="rms"))
    (logp.sum() + 0.1 * ent.sum()).backward()
    b = [t.detach().clone().requires_grad_() for t in (x, w, Wd)]
    logp2, ent2 = lm.lmhead_logps(lm.lmhead_norm(b[0], b[1], kind="rms"), b[2], tg, 64)
    (logp2.sum() + 0.1 * ent2.sum()).backward()
    torch.cuda.synchronize()
    assert torch.equal(logp, logp2) and torch.equal(ent, ent2)
    assert all(torch.equal(p.grad, q.grad) for p, q in zip(a, b))
    frozen = x.clone().requires_grad_()
    logp3, _ = lm.lmhead_logps(frozen, Wd, tg, 64, norm=lm.Norm(w, kind="rms"))
    logp3.sum().backward()
    assert w.grad is None and torch.isfinite(frozen.grad).all()


@pytest.mark.parametrize("N,V", [(180, 900), (700, 9000), (600, 70001)])   # few tokens; split; two blocks
def test_captured_step_replays(N, V):
    """Norm, distillation and both backward passes in one captured graph, on
    its own workspaces: every replay gives the eager bits, with eager work
    between the replays and new values in the same buffers."""
    import torch
    import cross_entropy_amd as lm
    H, K = 128, 9
    h, W, targets, ids, t, _ = _case(18, N, H, V, K, hard=True)
    x = dev(bf16_bits_to_f32(h))
    w = dev(np.linspace(0.5, 1.5, H).astype(np.float32))
    Wd, tg, idd, td = dev_bits(W), dev(targets), dev(ids), dev(t)
    gk, gl = (dev(a) for a in _g(7, N, True))
    ws = lm.distill_workspace_for(dev_bits(h), Wd, idd, 64, "bf16")
    wn = lm.norm_workspace_for(x)
    y = torch.empty(N, H, device="cuda", dtype=torch.bfloat16)
    mean, rstd, kl, logp, lse = (torch.empty(N, device="cuda") for _ in range(5))
    top = torch.empty(N, K, device="cuda")
    dh, dW = torch.empty_like(y), torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    dx, dw, db = torch.empty_like(x), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")

    def step():
        lm.lmhead_logps_norm_fwd(x, w, None, 1e-6, "layer", y, mean, rstd)
        lm.lmhead_logps_distill_fwd(y, Wd, tg, idd, td, None, 64, 1.0, kl, logp, lse, top, ws)
        lm.lmhead_logps_distill_bwd(y, Wd, tg, idd, td, None, 64, 1.0, logp, lse, top, gk, gl, dh, dW, 0, ws)
        lm.lmhead_logps_norm_bwd(x, w, "layer", mean, rstd, dh, dx, dw, db, 0, wn)

    outs = (y, mean, rstd, kl, logp, lse, top, dh, dW, dx, dw, db)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.mul_(1.1).add_(0.01 * i)
        for o in outs:
            o.fill_(float("nan"))
        ws.fill_(255)
        wn.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), i


@pytest.mark.parametrize("N,rows", [(40, 500), (300, 900)])
def test_two_streams_at_once(N, rows):
    """Calls on two streams with workspaces of their own, started together,
    give the lone calls' bits."""
    import torch
    import cross_entropy_amd as lm
    puts = [_put(*_case(20 + i, N, 128, 1300, 8, hard=True)) for i in range(2)]
    gk, gl = (dev(a) for a in _g(8, N, True))
    xs = [torch.randn(rows, 640, device="cuda") for _ in range(2)]

    def run(i):
        hd, Wd, tg, idd, td, tl = puts[i]
        kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
        out = (kl, logp, lse, top) + lm.distill_backward(hd, Wd, tg, idd, td, 64, logp, lse, top, gk, gl, tl)
        y, mean, rstd = lm.norm_forward(xs[i])
        return out + (y, mean, rstd) + lm.norm_backward(xs[i], None, mean, rstd, y, with_bias=True)

    lone = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        both = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                both.append(run(i))
        torch.cuda.synchronize()
        for a, b in zip(lone, both):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_distill_refuses_what_it_does_not_take():
    import torch
    import cross_entropy_amd as lm
    hd, Wd, tg, idd, td, _ = _put(*_case(19, 10, 64, 50, 4))
    ok = (hd, Wd, tg, idd, td, 8)
    lm.distill_forward(*ok)
    for i, bad, err in ((3, idd.long(), TypeError), (4, td.half(), TypeError), (4, td[:, :3], ValueError),
                        (3, idd[:9], ValueError), (3, idd.t().contiguous().t(), ValueError), (2, tg[:9], ValueError),
                        (2, tg.long(), TypeError), (0, hd.float(), TypeError), (1, Wd[:, :32], ValueError),
                        (4, td.cpu(), ValueError), (5, 0, lm.LmheadError)):
        args = list(ok)
        args[i] = bad
        with pytest.raises(err):
            lm.distill_forward(*args)
    with pytest.raises(lm.LmheadError):
        lm.distill_forward(*ok, temperature=0.0)
    with pytest.raises(ValueError):
        lm.distill_forward(*ok, torch.zeros(9, device="cuda"))
    kl, logp, lse, top = lm.distill_forward(*ok)
    with pytest.raises(lm.LmheadError):
        lm.distill_backward(*ok, None, lse, top, kl, logp)
    with pytest.raises(ValueError):
        lm.distill_backward(*ok, logp, lse, top[:, :3], kl)
    with pytest.raises(ValueError):
        lm.distill_backward(*ok, logp, lse, top, kl, accumulate=True)
    with pytest.raises(lm.LmheadError):
        lm.distill_backward(*ok, logp, lse, top, kl, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
