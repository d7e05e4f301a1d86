"""The front ends on the GPU: gradients under create_graph, calls without
tokens, the head's helpers given a stream."""
import pytest

from gpu_common import dev, dev_bits, log
from test_gpu_distill import _case

pytestmark = pytest.mark.gpu


def _inputs(N, H=128, V=300, K=4):
    import torch
    h, W, targets, ids, t, _ = _case(90 + N, max(N, 1), H, V, K, hard=True, pad=0.0)
    x = dev_bits(h).view(torch.bfloat16).float()[:N]
    w = torch.linspace(0.5, 1.5, H, device="cuda")
    leaves = [a.clone().requires_grad_() for a in (x, dev_bits(W).view(torch.bfloat16), w)]
    return leaves, dev(targets)[:N].contiguous(), dev(ids)[:N].contiguous(), dev(t)[:N].contiguous()


def _losses(lm, tg, ids, t):
    def head(x, W, w):
        logp, ent = lm.lmhead_logps(x, W, tg, 64, norm=lm.Norm(w, kind="rms"))
        return logp.sum() + 0.1 * ent.sum()

    def distill(x, W, w):
        kl, logp = lm.lmhead_distill(x, W, ids, t, 64, targets=tg, norm=lm.Norm(w))
        return kl.sum() - 0.1 * logp.sum()

    return head, distill


def test_second_backward_is_refused():
    import torch
    import cross_entropy_amd as lm
    leaves, tg, ids, t = _inputs(20)
    for loss in _losses(lm, tg, ids, t):
        log(f"[front ends] {loss.__name__}")
        want = torch.autograd.grad(loss(*leaves), leaves)
        total = loss(*leaves)
        got = torch.autograd.grad(total, leaves, create_graph=True)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        for g in got:
            with pytest.raises(RuntimeError, match="second backward"):
                (loss(*leaves) + g.float().pow(2).sum()).backward()


def test_front_ends_without_tokens():
    import torch
    import cross_entropy_amd as lm
    leaves, tg, ids, t = _inputs(0)
    for loss in _losses(lm, tg, ids, t):
        log(f"[front ends] no tokens, {loss.__name__}")
        got = torch.autograd.grad(loss(*leaves), leaves)
        torch.cuda.synchronize()
        assert got[0].shape == (0, 128) and all((g == 0).all() for g in got[1:])


def test_head_helpers_on_a_stream_of_their_own():
    """As tests/test_gpu_distill.py has it for the other helpers."""
    import torch
    import cross_entropy_amd as lm
    (x, W, _), tg, _, _ = _inputs(300, V=1300)
    h, W = x.detach().bfloat16(), W.detach()
    g = torch.linspace(-1, 1, 300, device="cuda")

    def run(stream):
        out = ()
        for T in (None, 0.7):
            logp, ent, lse = lm.forward(h, W, tg, 64, stream=stream, temperature=T)
            out += (logp, ent, lse)
            for ty in (torch.float32, torch.bfloat16):
                out += lm.backward(h, W, tg, 64, lse, ent, g, g, stream=stream, temperature=T, grad_dtype=ty)
        return out

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
