"""The vocabulary table's operators as they are used: a decode loop with beam
search, a training step with a tied table; captured and replayed, on two streams
at once, on a given stream, and within their buffers."""
import numpy as np
import pytest

import vocab_reference as R
from gpu_common import dev, dev_bits, log
from ops_reference import check
from synthetic import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


@pytest.mark.parametrize("B,G,V,steps", [(3, 4, 700, 5), (17, 5, 2001, 4), (40, 8, 1500, 3)])
def test_decode_loop(B, G, V, steps):
    """embed -> a toy recurrent state -> norm -> beam_step -> beam_reorder of the state, of a cache with lengths and of the
    token history. Every step's candidates are held to the definition on the step's own inputs, and every reordered
    tensor to what the parents say."""
    import torch
    import cross_entropy_amd as lm
    log(f"decode {B} {G} {V}")
    rng = np.random.default_rng(B)
    H, N, L = 128, B * G, 2 * steps
    Wbits = f32_to_bf16_bits((0.2 * rng.standard_normal((V, H))).astype(np.float32))
    W = dev_bits(Wbits).view(torch.bfloat16)
    norm = lm.Norm(weight=torch.rand(H, device="cuda") + 2.0, kind="rms")
    eos = 3
    tokens = torch.full((N,), 7, device="cuda", dtype=torch.int32)
    scores = torch.full((B, G), -float("inf"), device="cuda")
    scores[:, 0] = 0.0
    scores = scores.reshape(-1)
    ended = torch.full((N,), -1, device="cuda", dtype=torch.int32)
    state = torch.randn(B, 1, H, device="cuda").expand(B, G, H).reshape(N, H).contiguous()
    cache = torch.randint(0, 1000, (2, N, 2, L, 3), device="cuda", dtype=torch.int16)
    lengths = torch.randint(1, L, (B, 1), device="cuda", dtype=torch.int32).expand(B, G).reshape(-1).contiguous()
    history = torch.full((N, steps), -1, device="cuda", dtype=torch.int32)
    for step in range(steps):
        x = lm.lmhead_embed(W, tokens, 4.0, torch.float32)
        check(_np(x), *R.embed(bf16_bits_to_f32(Wbits), _np(tokens), 4.0, "f32"), "embed")
        state = (0.5 * state + x + 0.3 * torch.tanh(state.roll(1, 1))).contiguous()
        hidden, _, _ = lm.norm_forward(state, norm.weight, None, norm.eps, norm.kind, torch.bfloat16)
        top, ids, parents, lse = lm.beam_step(state, W, scores, G, ended=ended, norm=norm)
        ref = R.Beams(_np(hidden), bf16_bits_to_f32(Wbits), _np(scores), G, 2 * G, _np(ended))
        ref.check(_np(top), _np(ids), _np(parents), _np(lse), f"step {step}")
        take = slice(0, G)
        new, parent = ids[:, take].reshape(-1).contiguous(), parents[:, take].reshape(-1).contiguous()
        scores = top[:, take].reshape(-1).contiguous()
        before = [_np(t) for t in (cache, history, state)]
        state = lm.beam_reorder(state, parent, G, out=torch.empty_like(state))
        lm.beam_reorder(cache, parent, G, lengths=lengths, row_dim=1, length_dim=3)
        lm.beam_reorder(history, parent, G)
        p = _np(parent)
        assert np.array_equal(_np(cache), R.reorder(before[0], before[0], p, G, _np(lengths), 1, 3))
        assert np.array_equal(_np(history), R.reorder(before[1], before[1], p, G))
        assert np.array_equal(_np(state), R.reorder(before[2], before[2], p, G))
        history[:, step] = new
        ended = torch.where(new == eos, new, torch.where(ended[parent.long()] >= 0, ended[parent.long()], -1)).int()
        tokens = new
    assert (_np(history) >= 0).all()


def test_tied_table():
    """embed -> a layer -> norm -> the head's log-probs over the same table: autograd's gradient of the table is that of
    both uses, and so is the one that the embedding's backward adds to the head's in place."""
    import torch
    import cross_entropy_amd as lm
    g = torch.Generator(device="cuda").manual_seed(5)
    N, H, V = 300, 128, 500
    ids = torch.randint(-1, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    targets = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    W = (0.3 * torch.randn(V, H, device="cuda", generator=g)).bfloat16()
    weight = 0.5 + torch.rand(H, device="cuda", generator=g)

    def loss_of(table):
        x = lm.lmhead_embed(table, ids, 2.0, torch.float32)
        return lm.lmhead_logps(x, table, targets, 64, with_entropy=False, norm=lm.Norm(weight=weight, kind="rms")).sum()

    def exact(rows, head):
        x = torch.where((ids >= 0)[:, None], 2.0 * rows[ids.clamp(min=0).long()], 0.0)
        y = x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt() * weight.double()
        return torch.log_softmax(y @ head.t(), 1).gather(1, targets.long()[:, None]).sum()

    Wg = W.clone().requires_grad_()
    loss_of(Wg).backward()
    a, b = (W.double().requires_grad_() for _ in range(2))
    exact(a, b).backward()
    size = (a.grad + b.grad).norm()
    # bf16 hidden states and cotangents (2^-8 of each product's factors), and three roundings of a bf16 gradient
    bound = 8 * 2.0 ** -8
    assert (Wg.grad.double() - a.grad - b.grad).norm() <= bound * size
    # the same by hand, into the head's float32 gradient
    x = lm.embed_forward(W, ids, 2.0, torch.float32)
    h, mean, rstd = lm.norm_forward(x, weight, None, 1e-6, "rms", torch.bfloat16)
    logp, _, lse = lm.forward(h, W, targets, 64, with_entropy=False)
    dh, dW = lm.backward(h, W, targets, 64, lse, None, torch.ones(N, device="cuda"))
    dx, _, _ = lm.norm_backward(x, weight, mean, rstd, dh.bfloat16().float(), "rms", with_weight=False)
    head = dW.clone()
    lm.embed_backward(ids, dx, scale=2.0, dW=dW, accumulate=True)
    assert (dW.double() - a.grad - b.grad).norm() <= bound * size
    unused = torch.bincount(ids[ids >= 0].long(), minlength=V) == 0
    assert unused.any() and torch.equal(dW[unused], head[unused])


def _replayed(fill, call, outputs):
    """Captures call() and replays it on new inputs, with eager work and waits between, against eager results."""
    import torch
    fill(0)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(1, 5):
        fill(k)
        call()
        want = [o.clone() for o in outputs]
        for o in outputs:
            o.zero_()
        torch.cuda.synchronize()
        fill(k)
        graph.replay()
        (torch.randn(512, 512, device="cuda") @ torch.randn(512, 512, device="cuda")).sum()
        torch.cuda.synchronize()
        for o, w in zip(outputs, want):
            assert torch.equal(o, w), k
    return graph


@pytest.mark.parametrize("N,V,H", [(200, 900, 130), (5000, 900, 64), (300, 170000, 24)])
def test_captured_embedding(N, V, H):
    import torch
    import cross_entropy_amd as lm
    log(f"captured embedding {N} {V}")
    W, dy = torch.empty(V, H, device="cuda"), torch.empty(N, H, device="cuda")
    ids = torch.empty(N, device="cuda", dtype=torch.int32)
    y, dW, sums = torch.empty_like(dy), torch.empty_like(W), torch.empty_like(W)
    ws = [lm.embed_workspace_for(ids, W) for _ in range(2)]

    def fill(k):
        g = torch.Generator(device="cuda").manual_seed(k)
        W.normal_(generator=g)
        dy.normal_(generator=g)
        ids.copy_(torch.randint(-1, max(2, V // (1 + 100 * (k % 2))), (N,), device="cuda", generator=g))
        sums.fill_(1.0)

    def call():
        lm.lmhead_logps_embed_fwd(W, ids, 3.0, y)
        lm.lmhead_logps_embed_bwd(ids, dy, 3.0, dW, 0, ws[0])
        lm.lmhead_logps_embed_bwd(ids, dy, 3.0, sums, 2, ws[1])

    _replayed(fill, call, (y, dW, sums))
    check(_np(dW), *R.embed_grad(_np(ids), _np(dy), V, 3.0, None, "f32"), "dW")


@pytest.mark.parametrize("B,G,V", [(2, 4, 3000), (12, 8, 9000), (40, 8, 2500)])
def test_captured_beam_step_and_reorder(B, G, V):
    import torch
    import cross_entropy_amd as lm
    log(f"captured beam {B} {G} {V}")
    N, H, C = B * G, 64, 2 * G
    h, W = torch.empty(N, H, device="cuda", dtype=torch.bfloat16), torch.empty(V, H, device="cuda", dtype=torch.bfloat16)
    scores, lse = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    top, ids, parents = torch.empty(B, C, device="cuda"), *(torch.empty(B, C, device="cuda", dtype=torch.int32) for _ in range(2))
    states, out = torch.empty(2, N, 30, device="cuda"), torch.empty(2, N, 30, device="cuda")
    chosen = torch.empty(N, device="cuda", dtype=torch.int32)
    ws = lm.beam_workspace_for(h, W, G, C)

    def fill(k):
        g = torch.Generator(device="cuda").manual_seed(k)
        for t in (h, W, scores, states):
            t.normal_(generator=g)
        out.zero_()

    def call():
        lm.lmhead_logps_beam_step(h, W, scores, None, None, G, 1.0, top, ids, parents, lse, ws)
        chosen.copy_(parents[:, :G].reshape(-1))
        lm.lmhead_logps_beam_reorder(states, chosen, G, out, row_dim=1)

    _replayed(fill, call, (top, ids, parents, lse, out))
    R.Beams(_np(h), _np(W), _np(scores), G, C).check(_np(top), _np(ids), _np(parents), _np(lse), "replayed")


def test_two_streams_at_once():
    """Calls in flight on two streams, each with buffers of its own, give what they give alone."""
    import torch
    import cross_entropy_amd as lm

    def inputs(seed, N, V, H, G):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        ids = torch.randint(0, V // 50, (N,), device="cuda", generator=g, dtype=torch.int32)
        return r(N, H).bfloat16(), r(V, H).bfloat16(), r(N), ids, r(N, H), G

    def work(h, W, s, ids, dy, G, stream=None):
        out = list(lm.beam_step(h, W, s, G, stream=stream))
        out.append(lm.embed_backward(ids, dy, W.shape[0], stream=stream))
        out.append(lm.embed_forward(W, ids, 2.0, stream=stream))
        out.append(lm.beam_reorder(dy, out[2][:, :G].reshape(-1).contiguous() if stream is None else parents[id(h)], G,
                                   out=torch.empty_like(dy), stream=stream))
        return out

    a, b = inputs(1, 4000, 3000, 64, 8), inputs(2, 120, 40000, 128, 4)
    alone = [work(*x) for x in (a, b)]
    parents = {id(x[0]): w[2][:, :x[5]].reshape(-1).contiguous() for x, w in zip((a, b), alone)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [work(*x, stream=s) for x, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for w, g in zip(alone, got):
            for x, y in zip(w, g):
                assert torch.equal(x, y)


def _guarded(numel, dtype, offset=0):
    """A tensor of numel elements within a buffer, and a check that nothing around it changed."""
    import torch
    pad = 4096 // torch.empty(0, dtype=dtype).element_size()
    whole = torch.zeros(2 * pad + numel + offset, device="cuda", dtype=dtype)
    whole.view(torch.uint8).fill_(0xA5)
    part = whole[pad + offset:pad + offset + numel]

    def intact():
        head, tail = whole[:pad + offset].view(torch.uint8), whole[pad + offset + numel:].view(torch.uint8)
        return bool((head == 0xA5).all()) and bool((tail == 0xA5).all())
    return part, intact


@pytest.mark.parametrize("N,H,V,off", [(1, 1, 1, 0), (7, 33, 5, 1), (300, 1001, 77, 1), (2048, 64, 300, 0), (2049, 65, 300, 3),
                                       (5000, 40, 163841, 0), (4500, 257, 3, 1), (0, 9, 11, 1)])
def test_embedding_stays_within_its_buffers(N, H, V, off):
    """Outputs and workspaces of exactly the sizes asked for, outputs at odd element offsets."""
    import torch
    import cross_entropy_amd as lm
    log(f"guards {N} {H} {V}")
    ids = torch.randint(-1, V, (N,), device="cuda", dtype=torch.int32)
    for t in (torch.bfloat16, torch.float32):
        W, ok_W = _guarded(V * H, t, off)
        W.copy_(torch.randn(V * H, device="cuda"))
        y, ok_y = _guarded(N * H, t, off)
        dW, ok_dW = _guarded(V * H, t, off)
        ws, ok_ws = _guarded(lm.lmhead_logps_embed_workspace_bytes(N, H, V), torch.uint8)
        W, y, dW = W.view(V, H), y.view(N, H), dW.view(V, H)
        lm.lmhead_logps_embed_fwd(W, ids, 1.0, y)
        lm.lmhead_logps_embed_bwd(ids, y, 1.0, dW, 0, ws)
        check(_np(dW), *R.embed_grad(_np(ids), _np(y), V, 1.0, None, "f32" if t == torch.float32 else "bf16"), "dW")
        old = _np(dW)
        lm.lmhead_logps_embed_bwd(ids, y, 1.0, dW, 2, ws)
        check(_np(dW), *R.embed_grad(_np(ids), _np(y), V, 1.0, old, "f32" if t == torch.float32 else "bf16"), "dW added")
        assert ok_W() and ok_y() and ok_dW() and ok_ws()


@pytest.mark.parametrize("B,G,H,V,C", [(1, 1, 64, 1, 1), (5, 3, 64, 17, 7), (16, 4, 64, 5003, 8), (33, 3, 128, 1025, 64), (100, 2, 64, 24577, 5), (86, 3, 64, 300, 6)])
def test_beam_step_stays_within_its_buffers(B, G, H, V, C):
    import torch
    import cross_entropy_amd as lm
    log(f"guards beam {B} {G} {V}")
    N = B * G
    h, W = torch.randn(N, H, device="cuda").bfloat16(), torch.randn(V, H, device="cuda").bfloat16()
    scores = torch.randn(N, device="cuda")
    allowed = torch.randint(-2**31, 2**31, (N, (V + 31) // 32), device="cuda").int()
    for mask in (None, allowed):
        outs = [_guarded(n, t) for n, t in ((B * C, torch.float32), (B * C, torch.int32), (B * C, torch.int32), (N, torch.float32))]
        ws, ok_ws = _guarded(lm.lmhead_logps_beam_workspace_bytes(N, H, V, G, C), torch.uint8)
        top, ids, parents, lse = (o[0] for o in outs)
        top, ids, parents = (x.view(B, C) for x in (top, ids, parents))
        lm.lmhead_logps_beam_step(h, W, scores, None, mask, G, 1.0, top, ids, parents, lse, ws)
        R.Beams(_np(h), _np(W), _np(scores), G, C, None, None if mask is None else _np(mask)).check(
            _np(top), _np(ids), _np(parents), _np(lse), f"{B} {G} {V}")
        assert ok_ws() and all(o[1]() for o in outs)


def test_reorder_stays_within_its_buffers():
    import torch
    import cross_entropy_amd as lm
    for P, N, G, L, D, t in ((2, 6, 3, 7, 5, torch.uint8), (3, 40, 20, 9, 3, torch.int16), (1, 64, 64, 100, 1, torch.int32)):
        x, ok_x = _guarded(P * N * L * D, t, 1)
        x.copy_(torch.randint(0, 200, (P * N * L * D,), device="cuda"))
        x = x.view(P, N, L, D)
        first = torch.arange(N, device="cuda") // G * G
        parents = (first + torch.randint(0, G, (N,), device="cuda")).int()
        lengths = torch.randint(0, L + 1, (N,), device="cuda").int()
        before = _np(x)
        lm.beam_reorder(x, parents, G, lengths=lengths, row_dim=1)
        assert np.array_equal(_np(x), R.reorder(before, before, _np(parents), G, _np(lengths), 1)) and ok_x()
