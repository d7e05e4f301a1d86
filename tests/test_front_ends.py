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


class _On1:
    """The parts of a tensor on cuda:1 that the calls look at."""
    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, dtype, *shape):
        self.dtype, self.shape = dtype, torch.Size(shape)

    dim = lambda self: len(self.shape)                 # noqa: E731
    numel = lambda self: self.shape.numel()            # noqa: E731
    is_contiguous = lambda self: True                  # noqa: E731
    data_ptr = lambda self: 64                         # noqa: E731


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A launch on the default stream goes to the current device: every call
    makes its tensors' one current, and leaves the caller's as it was."""
    now, seen = [0], []

    class Device:
        def __init__(self, d):
            self.d = d.index

        def __enter__(self):
            self.back, now[0] = now[0], self.d

        def __exit__(self, *exc):
            now[0] = self.back

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    raws = ("fwd", "fwd_temp", "fwd_noalloc", "fwd_shard", "merge_shards", "bwd", "bwd_temp", "bwd_ex", "bwd_bf16",
            "bwd_shard", "distill_fwd", "distill_bwd", "norm_fwd", "norm_bwd")
    for name in raws:
        monkeypatch.setattr(lm._native, "raw_" + name, lambda *a, name=name: seen.append((name, now[0])) or 0)
    f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32
    h, W, ws = _On1(bf16, 4, 64), _On1(bf16, 9, 64), _On1(torch.uint8, 100)
    t, s, top, ids = _On1(i32, 4), _On1(f32, 4), _On1(f32, 4, 3), _On1(i32, 4, 3)
    dh, dW, v = _On1(f32, 4, 64), _On1(f32, 9, 64), _On1(f32, 64)
    out = dict(stream=0)
    lm.lmhead_logps_fwd(h, W, t, 8, s, s, s, ws, **out)
    lm.lmhead_logps_fwd_temp(h, W, t, 8, 0.7, s, s, s, ws, **out)
    lm.lmhead_logps_fwd_noalloc(h, W, t, 8, 0.7, s, s, s, **out)
    lm.lmhead_logps_fwd_shard(h, W, t, 0, 18, 8, 1.0, _On1(f32, 4, 4), ws, **out)
    lm.lmhead_logps_merge_shards(_On1(f32, 2, 4, 4), t, 18, 1.0, s, s, s, **out)
    lm.lmhead_logps_bwd(h, W, t, 8, s, s, s, s, dh, dW, ws, **out)
    lm.lmhead_logps_bwd_temp(h, W, t, 8, 0.7, s, s, s, s, dh, dW, ws, **out)
    lm.lmhead_logps_bwd_ex(h, W, t, 8, 0.7, s, s, s, s, dh, dW, 0, ws, **out)
    lm.lmhead_logps_bwd_bf16(h, W, t, 8, 0.7, s, s, s, s, h, W, 0, ws, **out)
    lm.lmhead_logps_bwd_shard(h, W, t, 0, 18, 8, 1.0, s, s, s, s, dh, dW, 0, ws, **out)
    lm.lmhead_logps_distill_fwd(h, W, t, ids, top, s, 8, 1.0, s, s, s, top, ws, **out)
    lm.lmhead_logps_distill_bwd(h, W, t, ids, top, s, 8, 1.0, s, s, top, s, s, dh, dW, 0, ws, **out)
    lm.lmhead_logps_norm_fwd(dh, v, v, 1e-6, "layer", dh, s, s, **out)
    lm.lmhead_logps_norm_bwd(dh, v, "layer", s, s, dh, dh, v, v, 0, ws, **out)
    assert sorted(seen) == sorted((name, 1) for name in raws) and now == [0]


def test_helpers_allocate_for_the_calls_stream(monkeypatch):
    """Outputs and workspaces of the helpers given a stream come from that
    stream's own pool: from the current stream's, a workspace freed on return
    could be handed out while the call still runs."""
    inside, made = [0], []

    class Pool:
        def __enter__(self):
            inside[0] += 1

        def __exit__(self, *exc):
            inside[0] -= 1

    def empty(*shape, dtype=None, device=None, **kw):
        made.append(inside[0])
        return _On1(dtype, *(shape[0] if isinstance(shape[0], tuple) else shape))

    monkeypatch.setattr(lm, "_allocating", lambda device, stream: Pool())
    monkeypatch.setattr(lm, "_enqueue", lambda dev, raw, *a: None)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(lm._native, "raw_workspace_bytes", lambda *a: 64)
    h, W, t, s = _On1(torch.bfloat16, 4, 64), _On1(torch.bfloat16, 9, 64), _On1(torch.int32, 4), _On1(torch.float32, 4)
    for temperature in (None, 0.7):
        lm.forward(h, W, t, 8, stream=7, temperature=temperature)
        for dtype in (torch.float32, torch.bfloat16):
            lm.backward(h, W, t, 8, s, s, s, stream=7, temperature=temperature, grad_dtype=dtype)
    assert len(made) == 2 * (4 + 2 * 3) and all(made)
