"""The autograd front ends on the host, the library's calls replaced by plain
torch forms: what the front ends add around them."""
import pytest
import torch

import cross_entropy_amd as lm


def _distill_forward(hidden, W, targets, ids, teacher, chunk_size, teacher_lse=None, temperature=1.0):
    z = hidden @ W.t()
    return z.pow(2).sum(1), None if targets is None else z.sum(1), z[:, 0], z


def _distill_backward(hidden, W, targets, ids, teacher, chunk_size, logp, lse, logp_top, g_kl, g_logp=None,
                      teacher_lse=None, temperature=1.0, grad_dtype=None):
    dz = 2 * g_kl[:, None] * (hidden @ W.t())
    if g_logp is not None:
        dz = dz + g_logp[:, None]
    return dz @ W, dz.t() @ hidden


def _head_forward(hidden, W, targets, chunk_size, with_entropy=True, temperature=None):
    z = hidden @ W.t()
    return z.pow(2).sum(1), z.sum(1) if with_entropy else None, z[:, 0]


def _head_backward(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent=None, temperature=None, grad_dtype=None):
    dz = 2 * g_logp[:, None] * (hidden @ W.t())
    if g_ent is not None:
        dz = dz + g_ent[:, None]
    return dz @ W, dz.t() @ hidden


def _norm_forward(x, weight=None, bias=None, eps=1e-6, kind="layer", out_dtype=None):
    return x * weight + bias, None, x.new_ones(len(x))


def _norm_backward(x, weight, mean, rstd, dy, kind, with_weight, with_bias, grad_dtype):
    return dy * weight, (dy * x).sum(0), dy.sum(0)


@pytest.fixture
def plain(monkeypatch):
    for f in (_distill_forward, _distill_backward, _norm_forward, _norm_backward):
        monkeypatch.setattr(lm, f.__name__[1:], torch.no_grad()(f))   # the library's results carry no graph


def _leaves(*shapes):
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(s, generator=gen).requires_grad_() for s in shapes]


def _distill(h, W):
    ids = torch.zeros(len(h), 1, dtype=torch.int32)
    kl, logp = lm.lmhead_distill(h, W, ids, ids.float(), 8, targets=ids[:, 0])
    return kl.sum() + logp.sum()


def _norm(x, w):
    return (lm.lmhead_norm(x, w, torch.zeros(len(w))) ** 2).sum()


def _once(loss, leaves):
    """First-order gradients, also under create_graph; a loss with a penalty on
    them is an error, not the gradient without the penalty, also where the
    incoming gradient is a constant."""
    want = torch.autograd.grad(loss(*leaves), leaves)
    total = loss(*leaves)
    got = torch.autograd.grad(total, leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(RuntimeError, match="second"):
        (total + sum(g.pow(2).sum() for g in got)).backward()


@pytest.mark.parametrize("loss,shapes", [(_distill, ((3, 4), (5, 4))), (_norm, ((3, 4), (4,)))])
def test_second_order_gradients_are_refused(plain, loss, shapes):
    _once(loss, _leaves(*shapes))


@pytest.mark.parametrize("with_entropy", [True, False])
def test_second_order_gradients_of_the_head_are_refused(monkeypatch, with_entropy):
    monkeypatch.setattr(lm, "forward", torch.no_grad()(_head_forward))
    monkeypatch.setattr(lm, "backward", torch.no_grad()(_head_backward))

    def head(h, W):
        out = lm.lmhead_logps(h, W, torch.zeros(len(h), dtype=torch.int32), 8, with_entropy=with_entropy)
        return out[0].sum() + out[1].sum() if with_entropy else out.sum()

    _once(head, _leaves((3, 4), (5, 4)))
