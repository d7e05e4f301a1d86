"""The distillation's kernels for few tokens where the other tests do not take
them: gradients added into, each count of row blocks, the second word of the
cotangent."""
import pytest

import ops_reference as R
from gpu_common import dev, log
from synthetic import bf16_bits_to_f32
from test_distill_words import WORDS, two_words, words_case
from test_gpu_distill import _case, _check, _forward_check, _g, _put

pytestmark = pytest.mark.gpu

ADD = [(20, 777), (50, 1003), (120, 900), (180, 1025), (250, 700)]   # each K of the products, a ragged vocabulary


def _forward(args):
    import cross_entropy_amd as lm
    hd, Wd, tg, idd, td, tl = _put(*args)
    kl, logp, lse, top = lm.distill_forward(hd, Wd, tg, idd, td, 64, tl)
    return (hd, Wd, tg, idd, td), tl, (logp, lse, top)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("N,V", ADD)
def test_few_tokens_add_into_gradients(t, N, V):
    """Added into, a gradient is the float32 sum of what the buffer held and of
    the gradient's own float32 value, rounded once: bit for bit."""
    import torch
    import cross_entropy_amd as lm
    H = 192                                  # no multiple of a wave's 128 columns, nor of a workgroup's 256
    log(f"[distill] add N={N} V={V} {t}")
    args = _case(40 + N, N, H, V, 7, hard=True)
    given, tl, (logp, lse, top) = _forward(args)
    gk, gl = (dev(a) for a in _g(41, N, True))
    ty = torch.float32 if t == "f32" else torch.bfloat16
    ws = lm.distill_workspace_for(given[0], given[1], given[3], 64, "bf16")
    own_h, own_W = lm.distill_backward(*given, 64, logp, lse, top, gk, gl, tl)      # float32, not added
    masked = dev(~R.Distill(bf16_bits_to_f32(args[0]), bf16_bits_to_f32(args[1]), *args[2:], 1.0).used)
    assert masked.any()
    for flags in (1, 2, 3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(flags)
        ph, pW = (torch.randn(s, H, device="cuda", generator=gen).to(ty) for s in (N, V))
        room_h = torch.cat([ph, torch.full((3, H), 7.0, device="cuda", dtype=ty)])   # rows behind, left as they were
        room_W = torch.cat([pW, torch.full((3, H), 7.0, device="cuda", dtype=ty)])
        dh, dW = room_h[:N], room_W[:V]
        lm.lmhead_logps_distill_bwd(*given, tl, 64, 1.0, logp, lse, top, gk, gl, dh, dW, flags, ws)
        torch.cuda.synchronize()
        want_h, want_W = own_h.to(ty), own_W.to(ty)
        if flags & 1:
            want_h = (ph.float() + own_h).to(ty)
            assert torch.equal(dh[masked], ph[masked])
        else:
            assert (dh[masked] == 0).all()
        if flags & 2:
            want_W = (pW.float() + own_W).to(ty)
        assert torch.equal(dh[~masked], want_h[~masked]), flags
        assert torch.equal(dW, want_W), flags
        assert (room_h[N:] == 7).all() and (room_W[V:] == 7).all()


@pytest.mark.parametrize("V", [50001, 90001, 120011, 151936, 200003])   # 2 to 5 row blocks a wave, and a second round
@pytest.mark.parametrize("N", [7, 24, 50])
def test_few_tokens_of_a_large_vocabulary(N, V):
    what = f"few N={N} V={V}"
    log(f"[distill] {what}")
    hard = N != 24
    _check(_case(N + V, N, 64, V, 9, t_type="f32", tail=N == 50, hard=hard), C=512, what=what)


@pytest.mark.parametrize("N,H,V,K", WORDS)
def test_few_tokens_keep_two_words(N, H, V, K, monkeypatch):
    """Up to 64 tokens the cotangent is held as its rounding to bf16 and what
    that left, rounded: the bound of two words, which one word does not keep
    (tests/test_distill_words.py)."""
    log(f"[distill] two words N={N} H={H} V={V} K={K}")
    two_words(monkeypatch, N, V)
    _check(words_case(N, H, V, K), grads=("f32",), what=f"two words N={N} V={V}")


@pytest.mark.parametrize("N", [3, 20, 50, 300])   # the kernels for few tokens at each tile of theirs, and the tiles
@pytest.mark.parametrize("V", [5, 70, 300])
def test_scores_of_a_small_temperature(N, V):
    """T = 2^-28: the scale to base 2 takes the stand-in for a missing row's
    logit beyond float32, which must not reach the rows that are there."""
    T, K = 2.0 ** -28, 3
    log(f"[distill] T=2^-28 N={N} V={V}")
    args = _case(70 + N + V, N, 64, V, K, T, hard=True, pad=0.0, lean=False)
    _forward_check(args, _put(*args), T, 64, f"T=2^-28 N={N} V={V}")


def test_front_end_gradients_in_a_captured_step():
    """lmhead_distill with norm=, forward and backward, captured with no eager
    graph of its leaves alive: every replay gives the eager gradients."""
    import torch
    import cross_entropy_amd as lm
    for N, V in ((40, 700), (300, 900)):
        log(f"[distill] captured front end N={N} V={V}")
        h, W, targets, ids, t, _ = _case(80, N, 128, V, 6, hard=True)
        hd, Wd, tg, idd, td, _ = _put(h, W, targets, ids, t, None)
        x, Wb = hd.view(torch.bfloat16).float(), Wd.view(torch.bfloat16)
        w = torch.linspace(0.5, 1.5, 128, device="cuda")

        def step(leaves):
            kl, logp = lm.lmhead_distill(leaves[0], leaves[1], idd, td, 64, tg, norm=lm.Norm(leaves[2], kind="rms"))
            return torch.autograd.grad(kl.sum() - 0.5 * logp.sum(), leaves)

        fresh = lambda: [a.clone().requires_grad_() for a in (x, Wb, w)]   # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(fresh())
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        leaves = fresh()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(leaves)
        for i in range(3):
            with torch.no_grad():
                leaves[0].mul_(1.2)
            for g in got:
                g.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            want = step([a.detach().clone().requires_grad_() for a in leaves])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want)), i
