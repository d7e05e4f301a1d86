"""Cases, plain forms and exact values of the vocabulary table's other uses around the head.

Five operators: the embedding lookup with its scale, the table's gradient from sorted tokens, one step of beam search on
the head's never-stored logits, and the reordering of beams' states, into another buffer or in place.
"""
import math
import random

import numpy as np
import torch

own = False

# ---- cases -------------------------------------------------------------------------------------------------------


def listed():
    return [
        # the token that was just decoded: latency alone
        dict(name="embed_token", op="embed_fwd", N=1, H=2560, V=151936, w="bf16", y="bf16", pad=0.0),
        # a ragged batch with an odd hidden size, a float32 table for a bf16 stream
        dict(name="embed_odd", op="embed_fwd", N=4099, H=1001, V=50257, w="f32", y="bf16", pad=0.05),
        # one context rank's share of a long row, into a float32 stream
        dict(name="embed_rank", op="embed_fwd", N=15237, H=4096, V=151936, w="bf16", y="f32", pad=0.0),
        # a micro-batch of short sequences, float32 gradient
        dict(name="embed_bwd_small", op="embed_bwd", N=256, H=256, V=4096, y="bf16", g="f32", add=False, pad=0.05),
        # one sequence of 4096 tokens, added to the gradient that the head has left for the tied table
        dict(name="embed_bwd_tied", op="embed_bwd", N=4096, H=2560, V=151936, y="bf16", g="bf16", add=True, pad=0.05),
        # a batch of 16 sequences of 4096 tokens
        dict(name="embed_bwd_batch", op="embed_bwd", N=65536, H=2560, V=151936, y="bf16", g="bf16", add=False, pad=0.05),
        # one request with four beams
        dict(name="beam_step_one", op="beam_step", B=1, beams=4, C=8, H=1024, V=50257, T=1.0, dead=0, ended=0.0, masked=False),
        # a serving batch of eight requests, a few beams ended
        dict(name="beam_step_serve", op="beam_step", B=8, beams=8, C=16, H=2560, V=151936, T=1.0, dead=0, ended=0.1, masked=False),
        # a large offline batch under a grammar's masks, its last requests padded
        dict(name="beam_step_batch", op="beam_step", B=64, beams=16, C=32, H=2560, V=151936, T=0.75, dead=3, ended=0.1, masked=True),
        # the token history of one request
        dict(name="reorder_history", op="reorder", B=1, beams=4, P=1, Q=1, L=512, D=1, t="i32", place=False, ragged=False),
        # keys and values of eight layers of a serving batch, each request as long as it is
        dict(name="reorder_cache", op="reorder", B=8, beams=8, P=16, Q=8, L=1024, D=128, t="bf16", place=True, ragged=True),
        # recurrent states of a large batch, into the other of two buffers
        dict(name="reorder_states", op="reorder", B=64, beams=16, P=24, Q=1, L=1, D=4096, t="f32", place=False, ragged=False),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "beam_step", "reorder"])
    if op.startswith("embed"):
        H = rng.choice([_log_uniform(rng, 64, 4096), 8 * _log_uniform(rng, 8, 512)])
        V = _log_uniform(rng, 1000, min(151936, 151936 * 2560 // H))
        N = _log_uniform(rng, 1, min(65536, 65536 * 2560 // H))
        pad = rng.choice([0.0, 0.05, 0.3])
        if op == "embed_fwd":
            return dict(op=op, N=N, H=H, V=V, w=rng.choice(["bf16", "f32"]), y=rng.choice(["bf16", "f32"]), pad=pad)
        return dict(op=op, N=N, H=H, V=V, y=rng.choice(["bf16", "f32"]), g=rng.choice(["bf16", "f32"]), add=rng.random() < 0.5, pad=pad)
    beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    if op == "beam_step":
        H = 64 * _log_uniform(rng, 4, 64)
        V = _log_uniform(rng, 1000, 151936)
        B = _log_uniform(rng, 1, max(1, min(1024, 1024 * 2560 * 151936 // (H * V)) // beams))
        return dict(op=op, B=B, beams=beams, C=rng.choice([beams, 2 * beams, beams + 1]), H=H, V=V, T=rng.choice([1.0, 1.0, 0.75, 1.5]),
                    dead=rng.choice([0, 0, 1]) if B > 1 else 0, ended=rng.choice([0.0, 0.1, 0.3]), masked=rng.random() < 0.3)
    B, Q = _log_uniform(rng, 1, 64), rng.choice([1, 2, 8])
    t = rng.choice(["bf16", "f32", "i32", "u8"])
    D = rng.choice([1, 64, 128, _log_uniform(rng, 1, 1000)])
    L = _log_uniform(rng, 1, 2048)
    P = _log_uniform(rng, 1, max(1, min(64, (1 << 30) // (B * beams * Q * L * D * _SIZE[t]))))
    if P * B * beams * Q * L * D * _SIZE[t] > 1 << 31:
        L = 1
    return dict(op=op, B=B, beams=beams, P=P, Q=Q, L=L, D=D, t=t, place=rng.random() < 0.5, ragged=L > 1 and rng.random() < 0.7)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "u8": torch.uint8}
_SIZE = {"bf16": 2, "f32": 4, "i32": 4, "u8": 1}

# ---- inputs ------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    """Inputs in HBM, and the buffers that a training or serving loop keeps."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"embed_fwd": _prepare_embed, "embed_bwd": _prepare_embed, "beam_step": _prepare_beam, "reorder": _prepare_reorder}[case["op"]](case, gen)


def _words(V, gen, *shape):
    """Token ids, frequent ones more often, in no order of frequency."""
    rank = torch.exp(torch.rand(*shape, device="cuda", generator=gen) * math.log(V))
    return (rank.to(torch.int64) * 7919 % V).to(torch.int32)


def _prepare_embed(case, gen):
    N, H, V = case["N"], case["H"], case["V"]
    ids = _words(V, gen, N)
    ids[N - int(case["pad"] * N):] = -1
    s = dict(case=case, ids=ids, scale=math.sqrt(H))
    if case["op"] == "embed_fwd":
        s["W"] = (0.02 * torch.randn(V, H, device="cuda", generator=gen)).to(_TYPES[case["w"]])
        s["y"] = torch.empty(N, H, device="cuda", dtype=_TYPES[case["y"]])
        return s
    s["dy"] = (0.01 * torch.randn(N, H, device="cuda", generator=gen)).to(_TYPES[case["y"]])
    s["dW"] = torch.empty(V, H, device="cuda", dtype=_TYPES[case["g"]])
    if case["add"]:  # what the head's backward pass left
        s["dW"].normal_(0.0, 0.1, generator=gen)
    return s


def _prepare_beam(case, gen):
    B, G, H, V = case["B"], case["beams"], case["H"], case["V"]
    N = B * G
    W = (0.02 * torch.randn(V, H, device="cuda", generator=gen)).to(torch.bfloat16)
    # the beams of a request are near one another, and each leans towards a few words
    hidden = 0.8 * torch.randn(B, 1, H, device="cuda", generator=gen).expand(B, G, H).reshape(N, H) + 0.6 * torch.randn(N, H, device="cuda", generator=gen)
    words = _words(V, gen, N, 6)
    for k in range(6):
        lean = (10.0 - 1.2 * k) * (0.6 + 0.4 * torch.rand(N, 1, device="cuda", generator=gen)) / (0.0004 * H)
        hidden += lean * W[words[:, k].long()].float()
    # scores of some thirty tokens so far, the best beam first
    gap = torch.rand(B, G, device="cuda", generator=gen) * 0.8
    scores = (-20.0 - 20.0 * torch.rand(B, 1, device="cuda", generator=gen) - gap.cumsum(1)).reshape(N).contiguous()
    if G > 2:  # a beam that was given up
        scores[torch.rand(N, device="cuda", generator=gen) < 0.02] = -math.inf
    scores[N - case["dead"] * G:] = -math.inf  # requests that pad the batch
    over = torch.rand(N, device="cuda", generator=gen) < case["ended"]
    ended = torch.where(over, 2, -1).to(torch.int32) if case["ended"] else None
    allowed = None
    if case["masked"]:
        # a grammar: some beams may go anywhere, most to a fraction of the words, a few nowhere
        share = torch.rand(N, 1, device="cuda", generator=gen)
        bits = torch.randint(-2**31, 2**31, (2, N, (V + 31) // 32), device="cuda", generator=gen, dtype=torch.int64).to(torch.int32)
        allowed = torch.where(share < 0.3, -1, torch.where(share < 0.7, bits[0], torch.where(share < 0.95, bits[0] & bits[1], 0))).to(torch.int32).contiguous()
    C = case["C"]
    return dict(case=case, hidden=hidden.to(torch.bfloat16), W=W, scores=scores, ended=ended, allowed=allowed,
                top_scores=torch.empty(B, C, device="cuda"), top_ids=torch.empty(B, C, device="cuda", dtype=torch.int32),
                top_parents=torch.empty(B, C, device="cuda", dtype=torch.int32), lse=torch.empty(N, device="cuda"))


def _prepare_reorder(case, gen):
    B, G, t = case["B"], case["beams"], _TYPES[case["t"]]
    shape = (case["P"], B * G, case["Q"], case["L"], case["D"])
    if t.is_floating_point:
        states, other = (torch.empty(shape, device="cuda", dtype=t).normal_(generator=gen) for _ in range(2))
    else:
        states, other = (torch.randint(0, 256 if t == torch.uint8 else 151936, shape, device="cuda", generator=gen, dtype=t) for _ in range(2))
    # the better beams have more children; children come in the order of their scores
    u = torch.rand(B, G, device="cuda", generator=gen)
    parents = (G * u * u).to(torch.int32).clamp_(0, G - 1).sort(1).values
    parents += G * torch.arange(B, device="cuda", dtype=torch.int32)[:, None]
    lengths = None
    if case["ragged"]:  # how many steps each request has so far
        lengths = (1 + (torch.rand(B, 1, device="cuda", generator=gen) * case["L"]).to(torch.int32)).clamp_(max=case["L"]).expand(B, G).reshape(-1).contiguous()
    return dict(case=case, states=states, parents=parents.reshape(-1).contiguous(), lengths=lengths, out=states if case["place"] else other)


# ---- one pass ----------------------------------------------------------------------------------------------------


def run(state):
    if own:
        return _framework(state)
    return {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "beam_step": _beam_step, "reorder": _reorder}[state["case"]["op"]](state)


def _framework(s):
    import cross_entropy_amd as lm

    case = s["case"]
    op = case["op"]
    if op == "embed_fwd":
        lm.lmhead_logps_embed_fwd(s["W"], s["ids"], s["scale"], s["y"])
        return dict(y=s["y"])
    if op == "reorder":
        lm.lmhead_logps_beam_reorder(s["states"], s["parents"], case["beams"], s["out"], lengths=s["lengths"], row_dim=1,
                                     length_dim=3 if s["lengths"] is not None else None)
        return dict(states=s["out"])
    if op == "embed_bwd":
        if "workspace" not in s:  # kept by a training loop, as its output buffers are
            s["workspace"] = lm.embed_workspace_for(s["ids"], s["dW"])
        lm.lmhead_logps_embed_bwd(s["ids"], s["dy"], s["scale"], s["dW"], lm._native.BWD_ACCUMULATE_DW if case["add"] else 0, s["workspace"])
        return dict(dW=s["dW"])
    if "workspace" not in s:
        s["workspace"] = lm.beam_workspace_for(s["hidden"], s["W"], case["beams"], case["C"])
    lm.lmhead_logps_beam_step(s["hidden"], s["W"], s["scores"], s["ended"], s["allowed"], case["beams"], case["T"], s["top_scores"],
                              s["top_ids"], s["top_parents"], s["lse"], s["workspace"])
    return dict(top_scores=s["top_scores"], top_ids=s["top_ids"], top_parents=s["top_parents"], lse=s["lse"])


def _embed_fwd(s):
    ids, V = s["ids"], s["W"].shape[0]
    live = (ids >= 0) & (ids < V)
    y = s["W"][ids.clamp(0, V - 1).long()].float() * s["scale"]
    return dict(y=torch.where(live[:, None], y, 0.0).to(s["y"].dtype))


def _embed_bwd(s):
    ids, dW = s["ids"], s["dW"]
    V, H = dW.shape
    live = (ids >= 0) & (ids < V)
    rows = torch.where(live[:, None], s["dy"].float(), 0.0)
    total = torch.zeros(V, H, device="cuda").index_add_(0, ids.clamp(0, V - 1).long(), rows) * s["scale"]
    if s["case"]["add"]:
        total += dW.float()
    return dict(dW=dW.copy_(total))


def _beam_step(s):
    # in 64 bits: which of two candidates that are next to one another is the better one is an output
    B, G, C, T = (s["case"][k] for k in ("B", "beams", "C", "T"))
    V = s["W"].shape[0]
    scores, ended, allowed = s["scores"].double(), s["ended"], s["allowed"]
    z = s["hidden"].double() @ s["W"].double().t() / T
    m = z.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    found = scores[:, None] + (z - lse)
    dead = scores == -math.inf
    if allowed is not None:
        v = torch.arange(V, device="cuda")
        found = torch.where((allowed[:, v >> 5] >> (v & 31)) & 1 != 0, found, -math.inf)
    if ended is not None:  # such a beam has one child, itself
        over = ended >= 0
        itself = torch.arange(V, device="cuda") == ended[:, None]
        found = torch.where(over[:, None], torch.where(itself, scores[:, None], -math.inf), found)
        dead = dead | over
    top, at = found.reshape(B, G * V).topk(C, dim=1)
    none = top == -math.inf
    first = G * torch.arange(B, device="cuda")[:, None]
    return dict(top_scores=top.float(), top_ids=torch.where(none, -1, at % V).int(), top_parents=torch.where(none, -1, at // V + first).int(),
                lse=torch.where(dead, 0.0, lse[:, 0]).float())


def _reorder(s):
    out = s["out"]
    moved = s["states"].index_select(1, s["parents"])
    if s["lengths"] is None:
        return dict(states=out.copy_(moved))
    steps = torch.arange(out.shape[3], device="cuda")
    used = steps < s["lengths"][s["parents"].long(), None]
    return dict(states=out.copy_(torch.where(used[None, :, None, :, None], moved, out)))


# ---- what a pass cannot do without -------------------------------------------------------------------------------


def _distinct(N, V):
    """How many words N draws are expected to hold: rank r comes with probability log((r + 1) / r) / log V."""
    r = np.arange(1, V, dtype=np.float64)
    return float((1.0 - (1.0 - np.log1p(1.0 / r) / math.log(V)) ** N).sum())


def work(case):
    if case["op"].startswith("embed"):
        N, H, V = case["N"], case["H"], case["V"]
        n = N - int(case["pad"] * N)
        words = _distinct(n, V)
        if case["op"] == "embed_fwd":
            return {"bytes": 4 * N + words * H * _SIZE[case["w"]] + N * H * _SIZE[case["y"]], "flops": N * H}
        # the rows of the words that occur are added to, or the whole table is written
        table = 2 * words if case["add"] else V
        return {"bytes": 4 * N + n * H * _SIZE[case["y"]] + table * H * _SIZE[case["g"]], "flops": 2 * n * H}
    B, G = case["B"], case["beams"]
    N = B * G
    if case["op"] == "beam_step":
        H, V = case["H"], case["V"]
        live = N - case["dead"] * G
        mask = 4 * live * ((V + 31) // 32) if case["masked"] else 0
        return {"bytes": 2 * (live + V) * H + mask + 12 * N + 12 * B * case["C"], "flops": 2 * live * H * V}
    rng = random.Random(0)
    read = written = 0
    for _ in range(200):  # the share of rows that are read and written
        parents = sorted(min(G - 1, int(G * rng.random() ** 2)) for _ in range(G))
        moved = [p for j, p in enumerate(parents) if p != j or not case["place"]]
        read, written = read + len(set(moved)) / 200, written + len(moved) / 200
    row = case["P"] * case["Q"] * (0.5 * (case["L"] + 1) if case["ragged"] else case["L"]) * case["D"] * _SIZE[case["t"]]
    return {"bytes": B * (read + written) * row + 4 * N, "flops": 0}


# ---- values in 64 bits -------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "embed_fwd":
        y = torch.zeros(case["N"], case["H"], device="cuda", dtype=f64)
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["V"])).flatten()
        y[at] = s["W"].index_select(0, s["ids"][at]).to(f64).mul(s["scale"])
        return dict(y=y)
    if case["op"] == "embed_bwd":
        # tokens in the order of their words; a word's sum is the difference of two running sums, taken a few columns at a time
        V, H = case["V"], case["H"]
        ids, order = s["ids"].long().sort(stable=True)
        order = order[(ids >= 0) & (ids < V)]
        ends = torch.bincount(s["ids"][order].long(), minlength=V).cumsum(0)
        out = s["dW"].to(f64) if case["add"] else torch.zeros(V, H, device="cuda", dtype=f64)
        for c in range(0, H, 256):
            sums = torch.zeros(order.numel() + 1, min(256, H - c), device="cuda", dtype=f64)
            sums[1:] = s["dy"][order, c:c + 256].to(f64).cumsum(0)
            upto = sums[ends]
            out[:, c:c + 256] += s["scale"] * torch.diff(upto, dim=0, prepend=sums[:1])
        return dict(dW=out)
    if case["op"] == "reorder":
        if not s["states"].is_floating_point():
            return None
        src, out = s["states"].to(f64), s["out"].to(f64)
        lengths = s["lengths"].tolist() if s["lengths"] is not None else None
        for j, p in enumerate(s["parents"].tolist()):
            n = lengths[p] if lengths is not None else case["L"]
            out[:, j, :, :n] = src[:, p, :, :n]
        return dict(states=out)
    # request by request: each beam's own log-probabilities, its best words by a stable sort, then the best of all
    B, G, C, V = case["B"], case["beams"], case["C"], case["V"]
    Wt = s["W"].to(f64).t()
    top_scores = torch.full((B, C), -math.inf, device="cuda", dtype=f64)
    lse = torch.zeros(B * G, device="cuda", dtype=f64)
    shift = torch.arange(32, device="cuda", dtype=torch.int32)
    for b in range(B):
        rows = slice(b * G, (b + 1) * G)
        z = (s["hidden"][rows].to(f64) @ Wt) * (1.0 / case["T"])
        total = torch.logsumexp(z, 1)
        logp = torch.log_softmax(z, 1)
        if s["allowed"] is not None:
            bits = ((s["allowed"][rows, :, None] >> shift) & 1).flatten(1)[:, :V]
            logp = logp.masked_fill(bits == 0, -math.inf)
        child = s["scores"][rows].to(f64)[:, None] + logp
        alive = ~torch.isneginf(s["scores"][rows])
        if s["ended"] is not None:
            for j, e in enumerate(s["ended"][rows].tolist()):
                if e >= 0:
                    child[j] = -math.inf
                    child[j, e] = s["scores"][b * G + j].to(f64)
                    alive[j] = False
        lse[rows] = torch.where(alive, total, torch.zeros_like(total))
        top_scores[b] = child.flatten().sort(descending=True, stable=True).values[:C]
    return dict(top_scores=top_scores, top_ids=None, top_parents=None, lse=lse)
