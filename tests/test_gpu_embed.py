"""The embedding and its gradient (lmhead_logps_embed_fwd / _bwd) through the
C ABI and the front end, against float64, within bounds derived from the
roundings (tests/vocab_reference.py)."""
import numpy as np
import pytest

import vocab_reference as R
from gpu_common import dev, log
from ops_reference import check
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _values(rng, shape, t):
    x = rng.standard_normal(shape).astype(np.float32)
    return bf16_bits_to_f32(f32_to_bf16_bits(x)) if t == "bf16" else x


def _put(x, t):
    import torch
    return dev(x).to(torch.bfloat16) if t == "bf16" else dev(x)


def _type(t):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[t]


def _ids(rng, N, V, heavy=0.3):
    ids = rng.integers(0, V, N).astype(np.int32)
    ids[rng.random(N) < heavy] = min(5, V - 1)          # a frequent word
    ids[rng.random(N) < 0.1] = -1
    if N > 3:
        ids[1], ids[2] = V, np.iinfo(np.int32).min      # others outside the vocabulary
    return ids


FWD = [(1, 2560, 1000), (1, 1, 1), (3, 7, 5), (37, 1001, 300), (1000, 64, 257), (700, 8, 50), (130, 4096, 77), (5000, 129, 999)]


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("y", ["bf16", "f32"])
@pytest.mark.parametrize("N,H,V", FWD)
def test_lookup(N, H, V, w, y):
    import cross_entropy_amd as lm
    log(f"embed_fwd {N} {H} {V} {w} {y}")
    rng = np.random.default_rng(N + H)
    W, ids = _values(rng, (V, H), w), _ids(rng, N, V)
    for scale in (1.0, 11.3137):
        got = lm.embed_forward(_put(W, w), dev(ids), scale, _type(y)).float().cpu().numpy()
        check(got, *R.embed(W, ids, scale, y), f"y {N} {H} {V}")


BWD = [(1, 2560, 300), (1, 1, 1), (3, 7, 5), (63, 100, 40), (64, 64, 3), (65, 64, 1), (257, 1001, 300), (1000, 513, 64),
       (1000, 8, 1000), (5000, 136, 5000), (20000, 40, 700), (4099, 600, 2)]


@pytest.mark.parametrize("y,g", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("N,H,V", BWD)
def test_gradient(N, H, V, y, g):
    import torch
    import cross_entropy_amd as lm
    log(f"embed_bwd {N} {H} {V} {y} {g}")
    rng = np.random.default_rng(N + H + V)
    ids, dy = _ids(rng, N, V), _values(rng, (N, H), y)
    dy[ids < 0] = np.nan                                # masked tokens' rows may hold anything
    scale = 0.75 if N % 2 else 50.0
    d_ids, d_dy = dev(ids), _put(dy, y)
    dW = torch.full((V, H), float("nan"), device="cuda", dtype=_type(g))
    got = lm.embed_backward(d_ids, d_dy, scale=scale, dW=dW).float().cpu().numpy()
    check(got, *R.embed_grad(ids, dy, V, scale, None, g), f"dW {N} {H} {V}")
    old = _values(rng, (V, H), g)
    into = _put(old, g)
    again = [lm.embed_backward(d_ids, d_dy, scale=scale, dW=into.clone(), accumulate=True) for _ in range(2)]
    check(again[0].float().cpu().numpy(), *R.embed_grad(ids, dy, V, scale, old, g), f"dW added {N} {H} {V}")
    assert torch.equal(again[0], again[1])              # nothing depends on timing


def test_gradient_without_tokens_and_of_masked_ones():
    import torch
    import cross_entropy_amd as lm
    for N in (0, 5, 200):
        ids = torch.full((N,), -1, device="cuda", dtype=torch.int32)
        dy = torch.full((N, 72), float("nan"), device="cuda")
        dW = lm.embed_backward(ids, dy, 300)
        assert dW.shape == (300, 72) and not dW.any()
        kept = torch.randn(300, 72, device="cuda")
        assert torch.equal(lm.embed_backward(ids, dy, dW=kept.clone(), accumulate=True), kept)
        assert not lm.embed_forward(kept, ids).any()


def test_one_word_for_all_and_each_its_own():
    """Every token the same word (one sum over all), every token another, and words in falling order."""
    import torch
    import cross_entropy_amd as lm
    rng = np.random.default_rng(8)
    N, H = 10007, 96
    dy = _values(rng, (N, H), "f32")
    for ids, V in ((np.full(N, 3, np.int32), 9), (rng.permutation(N).astype(np.int32), N), (np.arange(N, dtype=np.int32)[::-1].copy(), N)):
        got = lm.embed_backward(dev(ids), dev(dy), V).cpu().numpy()
        check(got, *R.embed_grad(ids, dy, V, 1.0, None, "f32"), "dW")
    torch.cuda.synchronize()


def test_large_vocabularies():
    """More words than 256 classes of counters hold."""
    import torch
    import cross_entropy_amd as lm
    rng = np.random.default_rng(2)
    for V in (163841, 524289, 3000001):
        N, H = 3000, 16
        ids = rng.integers(0, V, N).astype(np.int32)
        ids[::3] = ids[0]
        ids[1], ids[2] = 0, V - 1
        dy = _values(rng, (N, H), "f32")
        got = lm.embed_backward(dev(ids), dev(dy), V)
        rows = np.unique(ids)
        want, e = R.embed_grad(np.searchsorted(rows, ids), dy, len(rows), 1.0, None, "f32")
        at = torch.from_numpy(rows.astype(np.int64)).cuda()
        check(got[at].cpu().numpy(), want, e, f"dW {V}")
        got[at] = 0.0
        assert not got.any()


def test_many_tokens_added_into_large_vocabularies():
    """The sorted path's addition over 512 and more classes of words."""
    import torch
    import cross_entropy_amd as lm
    rng = np.random.default_rng(3)
    for V in (600001, 3000001):
        log(f"embed_bwd added, V {V}")
        N, H = 4000, 24
        ids = rng.integers(0, V, N).astype(np.int32)
        ids[::3] = ids[0]
        ids[1], ids[2] = 0, V - 1
        dy = _values(rng, (N, H), "f32")
        into = torch.full((V, H), 0.5, device="cuda")
        lm.embed_backward(dev(ids), dev(dy), dW=into, accumulate=True)
        rows = np.unique(ids)
        old = np.full((len(rows), H), 0.5, np.float32)
        want, e = R.embed_grad(np.searchsorted(rows, ids), dy, len(rows), 1.0, old, "f32")
        at = torch.from_numpy(rows.astype(np.int64)).cuda()
        check(into[at].cpu().numpy(), want, e, f"dW {V}")
        into[at] = 0.5
        assert bool((into == 0.5).all())


def test_rows_past_32_bits():
    """A table and a gradient whose last rows lie beyond 2^32 bytes."""
    import torch
    import cross_entropy_amd as lm
    V, H = 1100000, 2048
    W = torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    W[V - 1], W[V - 2] = 2.0, 3.0
    ids = torch.tensor([V - 1, 0, V - 2, V - 1], device="cuda", dtype=torch.int32)
    y = lm.embed_forward(W, ids, 0.5)
    assert [y[i].unique().tolist() for i in range(4)] == [[1.0], [0.0], [1.5], [1.0]]
    dW = lm.embed_backward(ids, torch.ones(4, H, device="cuda", dtype=torch.bfloat16), dW=W)
    assert [dW[i].unique().tolist() for i in (V - 1, V - 2, 0, 1, V - 3)] == [[2.0], [1.0], [1.0], [0.0], [0.0]]


def test_infinities_and_zeros_in_the_gradient():
    """IEEE sums: an infinity or a NaN of a live token reaches its word's row alone."""
    import cross_entropy_amd as lm
    rng = np.random.default_rng(4)
    N, H, V = 300, 40, 50
    ids = (np.arange(N) % V).astype(np.int32)
    dy = _values(rng, (N, H), "f32")
    dy[7, 3], dy[8, 4], dy[58, 4], dy[9] = np.inf, np.inf, -np.inf, np.nan
    got = lm.embed_backward(dev(ids), dev(dy), V).cpu().numpy()
    want, e = R.embed_grad(ids, np.nan_to_num(dy, nan=0.0, posinf=0.0, neginf=0.0), V, 1.0, None, "f32")
    want[7, 3], want[8, 4], want[9] = np.inf, np.nan, np.nan
    check(got, want, e, "dW")


@pytest.mark.parametrize("w,y", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("H", [1000, 1001])
def test_lookup_of_many_tokens(H, w, y):
    """y larger than the caches near the units hold (33 MB upwards), which is stored past them."""
    import torch
    import cross_entropy_amd as lm
    log(f"embed_fwd large {H} {w} {y}")
    rng = np.random.default_rng(H)
    N, V = 17000, 300
    W, ids, scale = _values(rng, (V, H), w), _ids(rng, N, V), 11.3137
    got = lm.embed_forward(_put(W, w), dev(ids), scale, _type(y)).double()
    table, e = (torch.from_numpy(x).cuda() for x in R.embed(W, np.arange(V, dtype=np.int32), scale, y))
    live = dev(((ids >= 0) & (ids < V)))[:, None]
    at = dev(np.where((ids >= 0) & (ids < V), ids, 0)).long()
    assert bool((torch.where(live, (got - table[at]).abs() - e[at], got.abs()) <= 0).all())


@pytest.mark.parametrize("y,g", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("H", [1000, 1001])
def test_gradient_of_many_tokens(H, y, g):
    """dy larger than every cache (270 MB upwards), which is loaded past them; the bound is that of R.embed_grad."""
    import torch
    import cross_entropy_amd as lm
    log(f"embed_bwd large {H} {y} {g}")
    rng = np.random.default_rng(H)
    N, V, scale = 136000 if y == "bf16" else 68000, 9000, 0.75
    ids = dev(_ids(rng, N, V, heavy=0.01))
    gen = torch.Generator(device="cuda").manual_seed(H)
    dy = torch.randn(N, H, device="cuda", generator=gen).to(_type(y))
    old = torch.randn(V, H, device="cuda", generator=gen).to(_type(g))
    live = (ids >= 0) & (ids < V)
    at = ids[live].long()
    total, size = (torch.zeros(V, H, device="cuda", dtype=torch.float64) for _ in range(2))
    total.index_add_(0, at, dy[live].double())
    size.index_add_(0, at, dy[live].double().abs())
    n = torch.bincount(at, minlength=V)[:, None]
    for add in (False, True):
        got = lm.embed_backward(ids, dy, scale=scale, dW=old.clone(), accumulate=add).double()
        want, e = scale * total, scale * size * (n + 1) * R.U
        if add:
            want = want + old.double()
            e = e + R.U * (want.abs() + e)
        e = e * (1 + R.HALF[g]) + R.HALF[g] * want.abs() + R.TINY
        assert bool(((got - want).abs() <= torch.where(n > 0, e, 0.0)).all()), add


def test_front_end_gradients():
    """lmhead_embed against autograd of its definition, and against differences."""
    import torch
    import cross_entropy_amd as lm
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, 60, (4, 9), device="cuda", generator=g, dtype=torch.int32)
    W = torch.randn(60, 33, device="cuda", generator=g, requires_grad=True)
    r = torch.randn(4, 9, 33, device="cuda", generator=g)
    y = lm.lmhead_embed(W, ids, 3.0)
    (y * r).sum().backward()
    W2 = W.detach().double().requires_grad_()
    ((3.0 * W2[ids.clamp(min=0).long()] * (ids >= 0)[..., None]) * r).sum().backward()
    assert torch.allclose(W.grad.double(), W2.grad, rtol=0, atol=40 * 2.0 ** -24 * 3.0 * 20)
    # linear in W: a difference is the derivative but for the roundings of y
    d = torch.randn(60, 33, device="cuda", generator=g)
    diff = ((lm.lmhead_embed(W.detach() + d, ids, 3.0) - y.detach()).double() * r).sum()
    size = (3.0 * (W.abs().max() + d.abs().max()) * r.abs().sum()).item()
    assert abs(diff.item() - (W.grad.double() * d).sum().item()) <= 64 * 2.0 ** -24 * size
    # bf16 table, float32 stream; an expanded gradient is taken too
    Wb = W.detach().bfloat16().requires_grad_()
    lm.lmhead_embed(Wb, ids, 1.0, torch.float32).sum().backward()
    n = torch.bincount(ids[ids >= 0].long(), minlength=60).float()
    assert torch.equal(Wb.grad.float(), n[:, None].expand(60, 33))
    assert Wb.grad.dtype == torch.bfloat16
    # a second backward is refused, and without tokens all is empty
    grad, = torch.autograd.grad((lm.lmhead_embed(W, ids) * r).sum(), W, create_graph=True)
    with pytest.raises(RuntimeError, match="second backward"):
        grad.sum().backward()
    none = lm.lmhead_embed(W, ids[:0])
    assert none.shape == (0, 9, 33)
    grad, = torch.autograd.grad(none.sum(), W)
    assert not grad.any()


def test_refused_tensors():
    import torch
    import cross_entropy_amd as lm
    W = torch.zeros(10, 16, device="cuda")
    ids = torch.zeros(4, device="cuda", dtype=torch.int32)
    with pytest.raises(TypeError):
        lm.embed_forward(W, ids.long())
    with pytest.raises(TypeError):
        lm.embed_forward(W.half(), ids)
    with pytest.raises(ValueError):
        lm.embed_forward(W.t(), ids)
    with pytest.raises(ValueError):
        lm.embed_forward(W, ids.cpu())
    with pytest.raises(ValueError):
        lm.lmhead_logps_embed_fwd(W, ids, 1.0, torch.empty(4, 15, device="cuda"))
    with pytest.raises(ValueError):
        lm.embed_backward(ids, torch.zeros(4, 16, device="cuda"))
    with pytest.raises(ValueError):
        lm.embed_backward(ids, torch.zeros(4, 16, device="cuda"), 10, accumulate=True)
    with pytest.raises(lm.LmheadError):
        lm.lmhead_logps_embed_bwd(ids, torch.zeros(4, 16, device="cuda"), 1.0, W, 0, torch.empty(16, device="cuda", dtype=torch.uint8))
    with pytest.raises(lm.LmheadError):
        lm.embed_forward(W, ids, float("inf"))
