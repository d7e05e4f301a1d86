"""The step of beam search (lmhead_logps_beam_step) and the reordering of states
(lmhead_logps_beam_reorder) through the C ABI and their helpers, against float64
(tests/vocab_reference.py)."""
import numpy as np
import pytest

import vocab_reference as R
from gpu_common import dev, dev_bits, log
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _case(seed, B, G, H, V, ended=0.0, masked=False, dead=0):
    rng = np.random.default_rng(seed)
    N = B * G
    W = f32_to_bf16_bits((0.1 * rng.standard_normal((V, H))).astype(np.float32))
    h = rng.standard_normal((N, H)) * 0.6 + np.repeat(rng.standard_normal((B, H)) * 0.8, G, 0)
    Wf = bf16_bits_to_f32(W)
    for k in range(4):
        h += (1.0 + rng.random((N, 1))) / (0.01 * H) * Wf[rng.integers(0, V, N)]
    scores = (-10 - 5 * rng.random((B, 1)) - np.cumsum(rng.random((B, G)), 1)).reshape(N).astype(np.float32)
    if G > 2:
        scores[rng.random(N) < 0.05] = -np.inf
    if dead:
        scores[N - dead * G:] = -np.inf
    e = None
    if ended:
        e = np.where(rng.random(N) < ended, rng.integers(0, V, N), -1).astype(np.int32)
    a = None
    if masked:
        a = rng.integers(-2**31, 2**31, (N, -(-V // 32)), dtype=np.int64)
        a &= rng.integers(-2**31, 2**31, a.shape, dtype=np.int64)
        a[rng.random(N) < 0.3] = -1
        a[rng.random(N) < 0.1] = 0                  # nowhere to go
        a = a.astype(np.int32)
    return f32_to_bf16_bits(h.astype(np.float32)), W, scores, e, a


def _run(case, G, C, T=1.0, **kw):
    import cross_entropy_amd as lm
    h, W, s, e, a = case
    out = lm.beam_step(dev_bits(h), dev_bits(W), dev(s), G, C, None if e is None else dev(e), None if a is None else dev(a), T, **kw)
    return [x.cpu().numpy() for x in out]


def _reference(case, G, C, T=1.0):
    h, W, s, e, a = case
    return R.Beams(bf16_bits_to_f32(h), bf16_bits_to_f32(W), s, G, C, e, a, T)


# rows of the streaming kernels (1, 16, 17, 33, 64, 65 to 256 of small vocabularies) and of the tiles; vocabularies that
# end inside a block, a section and a tile
SHAPES = [(1, 1, 64, 1, 1), (1, 1, 64, 2, 3), (1, 4, 128, 15, 8), (1, 4, 128, 16, 8), (1, 4, 256, 1003, 8), (2, 8, 64, 4096, 16), (17, 1, 192, 333, 2),
          (5, 5, 128, 5001, 6), (3, 16, 64, 777, 32), (1, 64, 128, 2000, 64), (8, 8, 192, 9999, 16), (22, 3, 128, 12289, 5), (9, 12, 128, 1000, 24), (16, 16, 64, 4100, 20),
          (16, 16, 64, 30011, 32), (65, 4, 128, 2049, 8), (130, 2, 64, 50257, 4), (60, 10, 320, 7001, 64)]


@pytest.mark.parametrize("B,G,H,V,C", SHAPES)
def test_step(B, G, H, V, C):
    log(f"beam_step {B} {G} {H} {V} {C}")
    case = _case(B + V, B, G, H, V)
    for T in (1.0, 0.7):
        _reference(case, G, C, T).check(*_run(case, G, C, T), f"{B} x {G}, H {H}, V {V}, C {C}, T {T}")


@pytest.mark.parametrize("B,G,H,V,C", [s for s in SHAPES if s[3] > 100][::2])
def test_step_with_masks_and_ended_beams(B, G, H, V, C):
    log(f"beam_step masked {B} {G} {H} {V} {C}")
    case = _case(B + V + 1, B, G, H, V, ended=0.2, masked=True, dead=1 if B > 1 else 0)
    _reference(case, G, C).check(*_run(case, G, C), f"{B} x {G}, H {H}, V {V}, C {C}")


def _exact_logits(rng, N, H, V):
    """Small whole numbers, whose logits are exact in any order."""
    h = rng.integers(-3, 4, (N, H)).astype(np.float32)
    W = rng.integers(-2, 3, (V, H)).astype(np.float32) / 16
    return f32_to_bf16_bits(h), f32_to_bf16_bits(W)


@pytest.mark.parametrize("N,V", [(4, 1000), (64, 700), (256, 5000), (320, 3001)])
def test_ties_go_to_the_lowest_row_and_word(N, V):
    """Equal logits within a row, rows that are alike, rows without a preference."""
    log(f"ties {N} {V}")
    rng = np.random.default_rng(N)
    G, C, H = 4, 12, 64
    h, W = _exact_logits(rng, N, H, V)
    W[V // 2:V // 2 + 200] = W[:200]                # words that are alike
    h[2::G] = h[1::G]                               # rows that are alike, with the same scores
    scores = np.tile(np.array([-1.0, -2.0, -2.0, -30.0], np.float32), N // G)
    h[:G] = 0                                       # a group without a preference
    case = (h, W, scores, None, None)
    _reference(case, G, C).check(*_run(case, G, C), "ties", exactly=True)


@pytest.mark.parametrize("G,V,C", [(8, 65000, 64), (64, 4000, 64), (32, 30000, 64)])
def test_best_words_in_a_few_places(G, V, C):
    """Most of the best words at places that fall to the same threads of the selection, or all with one beam of many."""
    log(f"few places {G} {V}")
    rng = np.random.default_rng(G)
    h = rng.standard_normal((G, 64)).astype(np.float32)
    W = (0.1 * rng.standard_normal((V, 64))).astype(np.float32)
    h[:, 0] = 1.0
    W[:, 0] = np.where(np.arange(V) // 128 % 128 < 79, 10.0, -10.0)
    scores = np.full(G, -1.0, np.float32) if G == 8 else np.where(np.arange(G) == 5, -1.0, -60.0).astype(np.float32)
    case = (f32_to_bf16_bits(h), f32_to_bf16_bits(W), scores, None, None)
    _reference(case, G, C).check(*_run(case, G, C), f"{G} {V}")


def test_words_and_parents_exactly():
    """Without near ties the very words and parents of 64-bit scores come out."""
    for seed, (B, G, H, V, C) in enumerate([(1, 4, 128, 2000, 8), (8, 8, 64, 3000, 16), (40, 8, 64, 2500, 16)]):
        case = _case(seed, B, G, H, V)
        r = _reference(case, G, C)
        gap = np.diff(-r.top, axis=1)
        got = _run(case, G, C)
        near = (gap < 4 * r.e_lse.max()).any(1)     # groups with near ties are left to the other tests
        for k in (0, 1, 2):
            want = (r.top.astype(np.float32), r.ids, r.parents)[k]
            if k:
                assert np.array_equal(got[k][~near], want[~near])
        assert (~near).sum() * 2 >= len(near)


def test_first_step_and_few_words():
    """One live beam among several; fewer words than candidates; no live beam at all."""
    case = list(_case(5, 3, 4, 64, 6))
    case[2] = np.array([0, -np.inf, -np.inf, -np.inf] * 2 + [-np.inf, np.nan, np.inf, -np.inf], np.float32)
    for C in (1, 6, 8, 64):
        _reference(case, 4, C).check(*_run(case, 4, C), f"C {C}")
    top, ids, parents, lse = _run(case, 4, 8)
    assert np.isneginf(top[2]).all() and (ids[2] == -1).all() and (parents[2] == -1).all() and (lse[8:] == 0).all()
    assert (parents[:2, :6] == [[0], [4]]).all()


def test_rows_that_hold_anything():
    """Given-up and ended rows may hold NaN; NaN and infinite logits leave their row without candidates; -inf words are none."""
    for V in (500, 40000):
        case = list(_case(11, 40, 2, 64, V))
        h, W, s, _, _ = case
        h = h.copy()
        e = np.full(80, -1, np.int32)
        nan, inf = f32_to_bf16_bits(np.array([np.nan, np.inf], np.float32))
        s[0], e[3] = -np.inf, 7
        h[0], h[3] = nan, nan
        e[5], s[5] = 8, -np.inf                     # ended and given up
        e[6] = V                                    # outside the vocabulary: not ended
        h[9, 0] = nan                               # a live row with a NaN, and one with infinities
        h[11] = inf
        case = (h, W, s, e, None)
        r = _reference(case, 2, 5)
        got = _run(case, 2, 5)
        r.check(*got, f"V {V}")
        assert (got[1][1][got[2][1] == 3] == 7).all()
        # a word of logit -inf in every row, and one of +inf in the rows that like it
        Wi = W.copy()
        Wi[3] = 0
        Wi[3, 0] = f32_to_bf16_bits(np.array([-np.inf], np.float32))[0]
        h2 = _case(11, 40, 2, 64, V)[0]
        h2[:, 0] = f32_to_bf16_bits(np.where(np.arange(80) % 5 == 0, -1.0, 1.0).astype(np.float32))
        case = (h2, Wi, s, None, None)
        r = _reference(case, 2, 5)
        r.check(*_run(case, 2, 5), f"-inf, V {V}")


def test_small_temperatures_and_large_logits():
    case = _case(3, 4, 4, 64, 3000)
    for T in (1e-3, 30.0):
        _reference(case, 4, 8, T).check(*_run(case, 4, 8, T), f"T {T}")
    h = f32_to_bf16_bits(1000 * bf16_bits_to_f32(case[0]))
    case = (h,) + case[1:]
    _reference(case, 4, 8).check(*_run(case, 4, 8), "large")


@pytest.mark.parametrize("B,G,H,V,C", [(3, 4, 64, 3000, 16), (1, 64, 64, 9000, 64), (24, 16, 64, 4000, 40), (40, 8, 128, 30000, 20)])
@pytest.mark.parametrize("far", [-1e4, -1e9, float(np.finfo(np.float32).min)])
def test_scores_far_apart(B, G, H, V, C, far):
    """Beams that a caller holds back by a very low score, in groups whose other beams have fewer words left than there
    are candidates: the best of the held back ones come next, by what 64 bits tell apart at that score."""
    log(f"far apart {B} {G} {V} {far}")
    h, W, scores, _, _ = _case(G + V, B, G, H, V)
    rng = np.random.default_rng(V)
    N = B * G
    scores = np.where(np.isfinite(scores), scores, -20).astype(np.float32)
    scores.reshape(B, G)[:, 1:] = far               # first steps: one beam, the others held back
    scores.reshape(B, G)[:, 2::3] *= 0.75           # at two distances
    a = np.zeros((N, -(-V // 32)), np.int32)
    some = rng.integers(0, a.shape[1], (N, 3))
    np.put_along_axis(a, some, rng.integers(0, 2**31, some.shape).astype(np.int32) & 0x00010001, 1)
    a.reshape(B, G, -1)[:, -1] = -1
    case = (h, W, scores, None, a)
    for T in (1.0, 0.5):
        _reference(case, G, C, T).check(*_run(case, G, C, T), f"{B} x {G} {V} {far} {T}")


def test_step_with_norm_and_workspaces():
    import torch
    import cross_entropy_amd as lm
    h, W, s, _, _ = _case(9, 4, 4, 128, 1000)
    x = torch.randn(16, 128, device="cuda") * 5
    norm = lm.Norm(weight=torch.rand(128, device="cuda") + 0.5, kind="rms")
    Wd, sd = dev_bits(W).view(torch.bfloat16), dev(s)
    a = lm.beam_step(x, Wd, sd, 4, norm=norm)
    y, _, _ = lm.norm_forward(x, norm.weight, None, norm.eps, "rms", torch.bfloat16)
    ws = lm.beam_workspace_for(y, Wd, 4, 8)
    ws.fill_(255)
    b = lm.beam_step(y, Wd, sd, 4, 8, workspace=ws)
    for k in range(4):
        assert torch.equal(a[k], b[k])
    assert a[0].shape == (4, 8)
    none = lm.beam_step(y[:0], Wd, sd[:0], 4)
    assert none[0].shape == (0, 8) and none[3].shape == (0,)
    with pytest.raises(ValueError):
        lm.beam_step(y, Wd, sd, 3)
    with pytest.raises(ValueError):
        lm.beam_step(y, Wd, sd[:8], 4)
    with pytest.raises(TypeError):
        lm.beam_step(y, Wd, sd.double(), 4)
    with pytest.raises(ValueError):
        lm.beam_step(y, Wd, sd, 4, allowed=torch.zeros(16, 31, device="cuda", dtype=torch.int32))
    with pytest.raises(lm.LmheadError):
        lm.beam_step(y, Wd, sd, 4, 65)
    with pytest.raises(lm.LmheadError):
        lm.beam_step(y, Wd, sd, 4, 8, workspace=ws[:64])


# ---- reordering


REORDER = [((8, 5), 0, None, 4, "int32"), ((12, 1), 0, None, 3, "uint8"), ((2, 8, 3, 17, 6), 1, 3, 4, "int16"), ((3, 6, 40, 2), 1, 2, 2, "float32"),
           ((8, 2, 33), 0, 2, 8, "uint8"), ((34, 7, 5), 0, 1, 17, "int16"), ((2, 64, 9, 10), 1, 2, 64, "int32"), ((1, 40, 300), 1, 2, 20, "uint8"),
           ((4, 16, 2, 64, 64), 1, 3, 16, "int16"), ((5, 4, 1000), 1, None, 2, "float32")]


@pytest.mark.parametrize("shape,row_dim,length_dim,G,t", REORDER)
@pytest.mark.parametrize("kind", ["mixed", "stay", "first", "reverse"])
def test_reorder(shape, row_dim, length_dim, G, t, kind):
    import cross_entropy_amd as lm
    log(f"reorder {shape} {row_dim} {length_dim} {G} {t} {kind}")
    rng = np.random.default_rng(len(shape) + G)
    N = shape[row_dim]
    states = rng.integers(0, 250, shape).astype(t)
    other = rng.integers(0, 250, shape).astype(t)
    first = np.arange(N) // G * G
    parents = {"mixed": first + rng.integers(0, G, N), "stay": np.arange(N), "first": first,
               "reverse": first + G - 1 - np.arange(N) % G}[kind].astype(np.int32)
    if kind == "mixed":
        parents[0] = -1
        parents[N - 1] = N
        if N > G:
            parents[1] = G                           # of another group
    lengths = None
    if length_dim is not None:
        L = shape[length_dim]
        lengths = rng.integers(0, L + 1, N).astype(np.int32)
        if kind == "mixed":
            lengths[first[-1]] = L + 9               # as the whole
            lengths[G - 1] = -3                      # as none
    a = dict(lengths=None if lengths is None else dev(lengths), row_dim=row_dim, length_dim=length_dim)
    into = lm.beam_reorder(dev(states), dev(parents), G, out=dev(other), **a).cpu().numpy()
    assert np.array_equal(into, R.reorder(states, other, parents, G, lengths, row_dim, length_dim))
    place = lm.beam_reorder(dev(states), dev(parents), G, **a).cpu().numpy()
    assert np.array_equal(place, R.reorder(states, states, parents, G, lengths, row_dim, length_dim))


@pytest.mark.parametrize("beams", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("L,D", [(257, 64), (251, 67)])
def test_reorder_of_large_states(beams, L, D):
    """States larger than the caches near the units hold (33 MB upwards), which are stored past them."""
    import torch
    import cross_entropy_amd as lm
    log(f"reorder large {beams} {L} {D}")
    gen = torch.Generator(device="cuda").manual_seed(beams)
    N, planes, heads = 128, 3, 7
    x = torch.randint(0, 250, (planes, N, heads, L, D), device="cuda", dtype=torch.uint8, generator=gen)
    other = torch.randint(0, 250, x.shape, device="cuda", dtype=torch.uint8, generator=gen)
    first = torch.arange(N, device="cuda") // beams * beams
    parents = (first + torch.randint(0, beams, (N,), device="cuda", generator=gen)).int()
    lengths = torch.randint(0, L + 1, (N,), device="cuda", generator=gen).int()
    for n in (None, lengths):
        took = x[:, parents.long()]
        short = None if n is None else (torch.arange(L, device="cuda")[None] >= n[parents.long()][:, None])[None, :, None, :, None]
        for onto in (other, x):
            want = took if n is None else torch.where(short, onto, took)
            state = x.clone()
            out = state if onto is x else other.clone()
            got = lm.beam_reorder(state, parents, beams, out=out, lengths=n, row_dim=1, length_dim=None if n is None else 3)
            assert torch.equal(got, want), (n is None, onto is x)


def test_reorder_at_odd_addresses():
    """States that begin at any byte, and runs of any length."""
    import torch
    import cross_entropy_amd as lm
    rng = np.random.default_rng(1)
    for off in (1, 3, 8):
        for L in (1, 15, 16, 17, 250):
            flat = rng.integers(0, 255, off + 2 * 6 * L).astype(np.uint8)
            parents = np.array([1, 1, 0, 5, 4, 4], np.int32)
            d = dev(flat)
            lm.beam_reorder(d[off:].view(2, 6, L), dev(parents), 3, row_dim=1)
            want = flat.copy()
            v = flat[off:].reshape(2, 6, L)
            want[off:] = R.reorder(v, v, parents, 3, row_dim=1).ravel()
            assert np.array_equal(d.cpu().numpy(), want), (off, L)
    torch.cuda.synchronize()


def test_reorder_past_32_bits():
    import torch
    import cross_entropy_amd as lm
    x = torch.zeros(3, 4, 600_000_000, device="cuda", dtype=torch.uint8)
    for p in range(3):
        for j in range(4):
            x[p, j, -1], x[p, j, 0] = 10 * p + j + 1, 100 + 10 * p + j
    parents = torch.tensor([2, 0, 0, 3], device="cuda", dtype=torch.int32)
    lm.beam_reorder(x, parents, 4, row_dim=1)
    assert x[:, :, -1].tolist() == [[10 * p + j + 1 for j in (2, 0, 0, 3)] for p in range(3)]
    assert x[:, :, 0].tolist() == [[100 + 10 * p + j for j in (2, 0, 0, 3)] for p in range(3)]


def test_reorder_refusals():
    import torch
    import cross_entropy_amd as lm
    x = torch.zeros(2, 8, 5, device="cuda")
    p = torch.zeros(8, device="cuda", dtype=torch.int32)
    for kw in (dict(row_dim=3), dict(row_dim=0), dict(row_dim=1, length_dim=2), dict(row_dim=1, lengths=p, length_dim=1),
               dict(row_dim=2, lengths=p), dict(row_dim=1, out=x[:1]), dict(row_dim=1, lengths=p[:4])):
        with pytest.raises(ValueError):
            lm.beam_reorder(x, p, 4, **kw)
    with pytest.raises(ValueError):
        lm.beam_reorder(x.transpose(0, 1), p, 4)
    with pytest.raises(TypeError):
        lm.beam_reorder(x, p.long(), 4, row_dim=1)
    with pytest.raises(TypeError):
        lm.beam_reorder(x, p, 4, out=x.double(), row_dim=1)
    both = torch.zeros(3, 8, 5, device="cuda")
    with pytest.raises(lm.LmheadError):
        lm.beam_reorder(both[:2], p, 4, out=both[1:], row_dim=1)
    with pytest.raises(lm.LmheadError):
        lm.beam_reorder(x, p, 5, row_dim=1)
