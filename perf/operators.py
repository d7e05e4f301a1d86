"""Cases, plain forms and exact values of the distillation head and the final norm.

Four operators: the forward and backward pass of the head's distillation loss (a teacher's top logits against the
student's never-stored logits), and the forward and backward pass of the norm in front of the head.
"""
import math

import torch

own = False

# ---- cases -------------------------------------------------------------------------------------------------------


def listed():
    return [
        # the final norm of one decoded token: latency alone
        dict(name="norm_fwd_token", op="norm_fwd", N=1, H=2560, kind="rms", x="bf16", y="bf16", w="bf16", bias=False),
        # a ragged batch with an odd hidden size, float32 stream
        dict(name="norm_fwd_odd", op="norm_fwd", N=4099, H=1001, kind="layer", x="f32", y="bf16", w="f32", bias=True),
        # one context rank's share of a long row
        dict(name="norm_fwd_rank", op="norm_fwd", N=15237, H=4096, kind="layer", x="bf16", y="bf16", w="bf16", bias=True),
        # a micro-batch of short sequences
        dict(name="norm_bwd_small", op="norm_bwd", N=256, H=256, kind="layer", x="bf16", y="bf16", w="f32", bias=True),
        # one sequence of 4096 tokens, float32 stream
        dict(name="norm_bwd_seq", op="norm_bwd", N=4096, H=2560, kind="rms", x="f32", y="bf16", w="f32", bias=False),
        # a batch of 16 sequences of 4096 tokens
        dict(name="norm_bwd_batch", op="norm_bwd", N=65536, H=2560, kind="layer", x="bf16", y="bf16", w="bf16", bias=True),
        # a few tokens scored against a teacher's top 20: the vocabulary table read once for them
        dict(name="distill_fwd_few", op="distill_fwd", N=7, H=2560, V=151936, K=20, chunk=512, T=1.0, teacher="f32",
             tail=True, hard=True, pad=0.0),
        # packed ragged rows, an odd vocabulary, a softened teacher
        dict(name="distill_fwd_ragged", op="distill_fwd", N=1357, H=1024, V=50257, K=50, chunk=512, T=2.0, teacher="bf16",
             tail=False, hard=False, pad=0.1),
        # one sequence of 4096 tokens at a 152k vocabulary
        dict(name="distill_fwd_seq", op="distill_fwd", N=4096, H=2560, V=151936, K=64, chunk=512, T=1.0, teacher="bf16",
             tail=False, hard=True, pad=0.05),
        # a small student
        dict(name="distill_bwd_tiny", op="distill_bwd", N=256, H=256, V=4096, K=8, chunk=128, T=1.0, teacher="f32",
             tail=False, hard=True, pad=0.05),
        # the training step of that sequence
        dict(name="distill_bwd_seq", op="distill_bwd", N=4096, H=2560, V=151936, K=64, chunk=512, T=1.0, teacher="bf16",
             tail=True, hard=True, pad=0.05),
        # one context rank's share of a long row
        dict(name="distill_bwd_rank", op="distill_bwd", N=15237, H=4096, V=151936, K=32, chunk=4096, T=2.0, teacher="f32",
             tail=False, hard=False, pad=0.05),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "distill_fwd", "distill_bwd"])
    if op.startswith("norm"):
        H = rng.choice([_log_uniform(rng, 64, 16384), 64 * _log_uniform(rng, 1, 128), 8 * _log_uniform(rng, 8, 1024)])
        N = _log_uniform(rng, 1, min(65536, 65536 * 2560 // H))
        x = rng.choice(["bf16", "f32"])
        return dict(op=op, N=N, H=H, kind=rng.choice(["layer", "rms"]), x=x, y="bf16" if x == "bf16" else rng.choice(["bf16", "f32"]),
                    w=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    H = 64 * _log_uniform(rng, 4, 64)
    V = _log_uniform(rng, 4000, 151936)
    most = 15237 * 4096 * 151936 if op == "distill_bwd" else 4096 * 2560 * 151936
    N = _log_uniform(rng, 1, min(16384, most // (H * V)))
    return dict(op=op, N=N, H=H, V=V, K=_log_uniform(rng, 1, 128), chunk=rng.choice([128, 512, 1024, 4096]),
                T=rng.choice([1.0, 1.0, 0.7, 2.0]), teacher=rng.choice(["bf16", "f32"]), tail=rng.random() < 0.5,
                hard=rng.random() < 0.5, pad=rng.choice([0.0, 0.05, 0.3]))


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6

# ---- inputs ------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    """Inputs in HBM, and the output buffers that a training or serving loop keeps."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    N, H = case["N"], case["H"]
    f32 = torch.float32
    if case["op"].startswith("norm"):
        xt, yt, wt = _TYPES[case["x"]], _TYPES[case["y"]], _TYPES[case["w"]]
        # a residual stream before the final norm: rows of different sizes, a few large channels, a small mean
        x = randn(N, H) * torch.exp(randn(N, 1)) + 0.3 * randn(1, H)
        x[:, :: max(1, H // 7)] *= 8.0
        s = dict(case=case, x=x.to(xt), weight=(1.0 + 0.2 * randn(H)).to(wt), bias=(0.1 * randn(H)).to(wt) if case["bias"] else None)
        del x
        mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        if case["op"] == "norm_fwd":
            s |= dict(y=torch.empty(N, H, device="cuda", dtype=yt), mean=mean if case["kind"] == "layer" else None, rstd=rstd)
            return s
        x = s["x"].to(f32)
        mu = x.mean(1) if case["kind"] == "layer" else torch.zeros(N, device="cuda")
        rstd = torch.rsqrt(((x - mu[:, None]) ** 2).mean(1) + EPS)
        dy = randn(N, H)
        dy[torch.rand(N, device="cuda", generator=gen) < 0.05] = 0.0  # masked tokens
        s |= dict(mean=mu if case["kind"] == "layer" else None, rstd=rstd, dy=dy.to(yt), dx=torch.empty(N, H, device="cuda", dtype=xt),
                  dweight=torch.empty(H, device="cuda", dtype=wt), dbias=torch.empty(H, device="cuda", dtype=wt) if case["bias"] else None)
        return s

    V, K = case["V"], case["K"]
    W = (0.02 * torch.randn(V, H, device="cuda", generator=gen)).to(torch.bfloat16)
    # the teacher's top ids, frequent words more often; its logits in falling order
    rank = torch.exp(torch.rand(N, K, device="cuda", generator=gen) * math.log(V))
    ids = (rank.to(torch.int64) * 7919 % V).to(torch.int32)
    teacher = 18.0 - 1.7 * torch.log1p(torch.arange(K, device="cuda", dtype=f32)) + 0.7 * randn(N, K)
    teacher = teacher.sort(dim=1, descending=True).values
    # the student already leans towards the teacher's first ids
    hidden = randn(N, H)
    scale = 1.0 / (0.0004 * H)
    for k in range(min(K, 4)):
        hidden += (9.0 - 1.5 * k) * scale * W[ids[:, k].long()].to(f32)
    hidden = hidden.to(torch.bfloat16)
    if K > 1:
        # rows for which the teacher gave fewer entries, and entries that it forbids
        short = torch.rand(N, 1, device="cuda", generator=gen) < 0.2
        kept = 1 + (torch.rand(N, 1, device="cuda", generator=gen) * K).to(torch.int64)
        ids = torch.where(short & (torch.arange(K, device="cuda")[None] >= kept), -1, ids)
        teacher[:, 1:][torch.rand(N, K - 1, device="cuda", generator=gen) < 0.01] = -math.inf
    targets = ids[:, 0].clone()
    other = torch.randint(0, V, (N,), device="cuda", generator=gen, dtype=torch.int32)
    targets = torch.where(torch.rand(N, device="cuda", generator=gen) < 0.3, other, targets)
    padded = torch.arange(N, device="cuda") >= N - int(case["pad"] * N)
    ids[padded] = -1
    targets[padded] = -1
    teacher = teacher.to(_TYPES[case["teacher"]])
    tail = None
    if case["tail"]:  # the teacher's whole log-sum-exp, a little more than its top entries give
        tail = torch.logsumexp(teacher.to(f32) / case["T"], dim=1) + 0.2 * torch.rand(N, device="cuda", generator=gen)
    s = dict(case=case, hidden=hidden, W=W, targets=targets if case["hard"] else None, ids=ids.contiguous(), teacher=teacher,
             teacher_lse=tail, logp=torch.zeros(N, device="cuda") if case["hard"] else None, lse=torch.empty(N, device="cuda"),
             logp_top=torch.empty(N, K, device="cuda"))
    if case["op"] == "distill_fwd":
        s |= dict(kl=torch.empty(N, device="cuda"))
        return s
    Wf = W.to(f32)
    for r in range(0, N, 2048):  # the forward pass's values
        z = hidden[r:r + 2048].to(f32) @ Wf.t() / case["T"]
        lse = torch.logsumexp(z, dim=1)
        i = ids[r:r + 2048]
        top = z.gather(1, i.clamp(0, V - 1).long()) - lse[:, None]
        s["logp_top"][r:r + 2048] = torch.where(i >= 0, top, 0.0)
        s["lse"][r:r + 2048] = torch.where(padded[r:r + 2048], 0.0, lse)
        if case["hard"]:
            t = targets[r:r + 2048]
            s["logp"][r:r + 2048] = torch.where(t >= 0, z.gather(1, t.clamp(0, V - 1).long()[:, None])[:, 0] - lse, 0.0)
    s |= dict(g_kl=0.5 + torch.rand(N, device="cuda", generator=gen), g_logp=-0.3 * torch.rand(N, device="cuda", generator=gen) if case["hard"] else None,
              dh=torch.empty(N, H, device="cuda", dtype=torch.bfloat16), dW=torch.empty(V, H, device="cuda", dtype=torch.bfloat16))
    return s


# ---- one pass ----------------------------------------------------------------------------------------------------


def run(state):
    if own:
        return _framework(state)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "distill_fwd": _distill_fwd, "distill_bwd": _distill_bwd}[state["case"]["op"]](state)


def _framework(s):
    import cross_entropy_amd as lm

    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        lm.lmhead_logps_norm_fwd(s["x"], s["weight"], s["bias"], EPS, case["kind"], s["y"], s["mean"], s["rstd"])
        return _some(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    if "workspace" not in s:  # kept by a training loop, as its output buffers are
        if op == "norm_bwd":
            s["workspace"] = lm.norm_workspace_for(s["x"])
        else:
            s["workspace"] = lm.distill_workspace_for(s["hidden"], s["W"], s["ids"], case["chunk"], "bf16" if op == "distill_bwd" else False)
    if op == "norm_bwd":
        lm.lmhead_logps_norm_bwd(s["x"], s["weight"], case["kind"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dweight"], s["dbias"], 0,
                                 s["workspace"])
        return _some(dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])
    given = (s["hidden"], s["W"], s["targets"], s["ids"], s["teacher"], s["teacher_lse"], case["chunk"], case["T"])
    if op == "distill_fwd":
        lm.lmhead_logps_distill_fwd(*given, s["kl"], s["logp"], s["lse"], s["logp_top"], s["workspace"])
        return _some(kl=s["kl"], logp=s["logp"], lse=s["lse"], logp_top=s["logp_top"])
    lm.lmhead_logps_distill_bwd(*given, s["logp"], s["lse"], s["logp_top"], s["g_kl"], s["g_logp"], s["dh"], s["dW"], 0,
                                s["workspace"])
    return dict(dh=s["dh"], dW=s["dW"])


def _some(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _norm_fwd(s):
    x = s["x"].float()
    layer = s["case"]["kind"] == "layer"
    mean = x.mean(1) if layer else None
    c = x - mean[:, None] if layer else x
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return _some(y=y.to(s["y"].dtype), mean=mean, rstd=rstd)


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    layer = s["case"]["kind"] == "layer"
    xhat = (x - s["mean"][:, None] if layer else x) * rstd
    g = dy * s["weight"].float()
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    wt = s["weight"].dtype
    dweight = (dy * xhat).sum(0).to(wt)
    dbias = dy.sum(0).to(wt) if s["bias"] is not None else None
    return _some(dx=(dx * rstd).to(s["x"].dtype), dweight=dweight, dbias=dbias)


def _teacher(s):
    """log q and q over the entries [N, K]; an entry outside the vocabulary has q = 0."""
    ids, V, T = s["ids"], s["W"].shape[0], s["case"]["T"]
    live = (ids >= 0) & (ids < V)
    t = torch.where(live, s["teacher"].float() / T, -math.inf)
    if s["teacher_lse"] is not None:
        logq = t - s["teacher_lse"][:, None]
    else:
        m = t.amax(1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        logq = t - (m + torch.log(torch.exp(t - m).sum(1, keepdim=True)))
    some = t > -math.inf
    return live, torch.where(some, logq, 0.0), torch.where(some, torch.exp(logq), 0.0)


def _distill_fwd(s):
    T, V = s["case"]["T"], s["W"].shape[0]
    z = s["hidden"].float() @ s["W"].float().t() / T
    m = z.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
    live, logq, q = _teacher(s)
    top = torch.where(live, z.gather(1, s["ids"].clamp(0, V - 1).long()) - lse[:, None], 0.0)
    kl = (q * (logq - top)).sum(1)
    used = live.any(1)
    logp = None
    if s["targets"] is not None:
        hard = (s["targets"] >= 0) & (s["targets"] < V)
        used = used | hard
        logp = torch.where(hard, z.gather(1, s["targets"].clamp(0, V - 1).long()[:, None])[:, 0] - lse, 0.0)
    return _some(kl=kl, logp=logp, lse=torch.where(used, lse, 0.0), logp_top=top)


def _distill_bwd(s):
    T, V = s["case"]["T"], s["W"].shape[0]
    h, W = s["hidden"].float(), s["W"].float()
    live, _, q = _teacher(s)
    gq = s["g_kl"][:, None] * q
    coef = gq.sum(1)
    used = live.any(1)
    if s["targets"] is not None:
        hard = (s["targets"] >= 0) & (s["targets"] < V)
        used = used | hard
        g_hard = torch.where(hard, s["g_logp"], 0.0)
        coef = coef - g_hard
    coef = torch.where(used, coef, 0.0)
    dz = torch.exp(h @ W.t() / T - s["lse"][:, None])
    dz = torch.where(used[:, None], dz, 0.0) * coef[:, None]
    dz.scatter_add_(1, s["ids"].clamp(0, V - 1).long(), -gq)
    if s["targets"] is not None:
        dz.scatter_add_(1, s["targets"].clamp(0, V - 1).long()[:, None], g_hard[:, None])
    dz /= T
    return dict(dh=(dz @ W).to(torch.bfloat16), dW=(dz.t() @ h).to(torch.bfloat16))


# ---- what a pass cannot do without -------------------------------------------------------------------------------


def work(case):
    N, H = case["N"], case["H"]
    size = {"bf16": 2, "f32": 4}
    if case["op"].startswith("norm"):
        x, y, w = size[case["x"]], size[case["y"]], size[case["w"]]
        stats = 4 * N * (2 if case["kind"] == "layer" else 1)
        vectors = w * H * (2 if case["bias"] else 1)
        if case["op"] == "norm_fwd":
            return {"bytes": N * H * (x + y) + vectors + stats, "flops": 8 * N * H}
        return {"bytes": N * H * (2 * x + y) + vectors + w * H + stats, "flops": 14 * N * H}
    V, K = case["V"], case["K"]
    read = 2 * (N + V) * H + N * K * (4 + size[case["teacher"]]) + 4 * N * (int(case["hard"]) + int(case["tail"]))
    if case["op"] == "distill_fwd":
        return {"bytes": read + 4 * N * (2 + K + int(case["hard"])), "flops": 2 * N * V * H}
    # two products for the gradients, and the logits, which are not kept, once more
    return {"bytes": read + 4 * N * (2 + K + int(case["hard"])) + 2 * (N + V) * H, "flops": 6 * N * V * H}


# ---- values in 64 bits -------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"].startswith("norm"):
        x = s["x"].to(f64).requires_grad_()
        w = s["weight"].to(f64).requires_grad_()
        b = (s["bias"].to(f64) if s["bias"] is not None else torch.zeros_like(w, requires_grad=False)).detach().requires_grad_()
        if case["op"] == "norm_fwd":
            with torch.no_grad():
                var, mean = torch.var_mean(x, dim=1, unbiased=False)
                if case["kind"] == "rms":
                    var, mean = x.pow(2).mean(1), torch.zeros_like(mean)
                std = (var + EPS).sqrt()
                y = torch.addcmul(b, (x - mean[:, None]) / std[:, None], w)
            return _some(y=y, mean=mean if case["kind"] == "layer" else None, rstd=1 / std)
        # the gradient of sum(y dy), the statistics being functions of x
        out = None
        dx = torch.empty_like(x, requires_grad=False)
        dw, db = torch.zeros_like(w, requires_grad=False), torch.zeros_like(w, requires_grad=False)
        for r in range(0, case["N"], 8192):
            xr = s["x"][r:r + 8192].to(f64).requires_grad_()
            c = xr - xr.mean(1, keepdim=True) if case["kind"] == "layer" else xr
            out = (c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * w + b)
            gx, gw, gb = torch.autograd.grad((out * s["dy"][r:r + 8192].to(f64)).sum(), (xr, w, b))
            dx[r:r + 8192], dw, db = gx, dw + gw, db + gb
        return _some(dx=dx, dweight=dw, dbias=db if s["bias"] is not None else None)

    N, V, K, T = case["N"], case["V"], case["K"], case["T"]
    W = s["W"].to(f64)
    back = case["op"] == "distill_bwd"
    dW = torch.zeros_like(W) if back else None
    rows = []
    for r in range(0, N, 1024):
        part = slice(r, r + 1024)
        h = s["hidden"][part].to(f64)
        ids = s["ids"][part].long()
        live = (ids >= 0) & (ids < V)
        z = ((h @ W.t()) / T).requires_grad_(back)
        lse = torch.logsumexp(z, dim=1)
        logs = z - lse[:, None]
        t = s["teacher"][part].to(f64) / T
        given = live & ~torch.isneginf(t)
        e = torch.where(given, t, 0.0)
        if s["teacher_lse"] is not None:
            q = torch.exp(e - s["teacher_lse"][part].to(f64)[:, None]) * given
        else:
            big = torch.where(given, t, -1e300).max(dim=1, keepdim=True).values
            q = torch.exp(torch.where(given, t - big, 0.0)) * given
            q = q / q.sum(1, keepdim=True).clamp_min(1e-300)
        top = torch.where(live, logs.gather(1, ids.clamp(0, V - 1)), 0.0)
        kl = (torch.special.xlogy(q, q) - q * top).sum(1)
        used, logp = live.any(1), None
        if s["targets"] is not None:
            target = s["targets"][part].long()
            hard = (target >= 0) & (target < V)
            used = used | hard
            logp = torch.where(hard, logs.gather(1, target.clamp(0, V - 1)[:, None])[:, 0], 0.0)
        if not back:
            rows.append(_some(kl=kl, logp=logp, lse=torch.where(used, lse, 0.0), logp_top=top))
            continue
        loss = (s["g_kl"][part].to(f64) * kl).sum()
        if logp is not None:
            loss = loss + (s["g_logp"][part].to(f64) * logp).sum()
        dz = torch.autograd.grad(loss, z)[0] / T
        rows.append(dict(dh=dz @ W))
        dW += dz.t() @ h
        del z, logs, dz, loss
    found = {k: torch.cat([x[k] for x in rows]) for k in rows[0]}
    return found | {"dW": dW} if back else found
