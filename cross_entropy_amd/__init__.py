"""MI355X (gfx950) fused LM-head log-prob and entropy head.

Per token: logits z = h W^T over the whole vocabulary (never stored), lse,
logp = z[target] - lse and entropy = lse - sum softmax(z) z, and the
backward into dh and dW. All of it runs in the HIP library
``liblmhead_logps.so`` (C ABI in ``include/lmhead_logps.h``); this module
only checks torch tensors and passes their device pointers and the current
HIP stream. PyTorch provides device memory and streams, nothing else.

Entry points mirror the C ABI:
    lmhead_logps_workspace_bytes(N, H, V, chunk_size, with_backward)
    lmhead_logps_fwd(hidden, W, targets, chunk_size, logp, entropy, lse, workspace)
    lmhead_logps_bwd(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent,
                     dh, dW, workspace)
    lmhead_logps_fwd_temp / lmhead_logps_bwd_temp   (the same with a temperature
                     after chunk_size: the head scores the logits divided by it)
    lmhead_logps_bwd_ex  (tempered backward that can add into dh / dW)
    lmhead_logps_bwd_bf16  (the same writing bf16 dh / dW: float32 sums in the
                         workspace, each element rounded once)
    lmhead_logps_fwd_shard / lmhead_logps_merge_shards / lmhead_logps_bwd_shard
                         (the head over vocabulary shards, partials merged by log-sum-exp)
    lmhead_logps_fwd_noalloc  (tempered forward without a workspace, for callers
                         that cannot allocate; its scratch is a fixed device array)
    lmhead_logps_distill_fwd / lmhead_logps_distill_bwd  (KL to a teacher's top
                         logits, and the log-prob of a hard target beside it)
    lmhead_logps_norm_fwd / lmhead_logps_norm_bwd  (the layer or RMS norm in
                         front of the head)
    lmhead_logps_embed_fwd / lmhead_logps_embed_bwd  (the vocabulary table as an
                         embedding, and its gradient from sorted tokens)
    lmhead_logps_beam_step / lmhead_logps_beam_reorder  (beam search's step over
                         the head's never-held logits, and its states' reordering)
with allocating helpers for the last four pairs (``distill_forward``,
``distill_backward``, ``norm_forward``, ``norm_backward``, ``embed_forward``,
``embed_backward``, ``beam_step``, ``beam_reorder``) and autograd front ends
(``lmhead_distill``, ``lmhead_norm``, ``lmhead_embed``);
two allocating helpers for the head, ``forward`` and ``backward`` (``temperature=``
selects the tempered calls, ``dh=`` / ``dW=`` with ``accumulate=`` add into
caller buffers), and ``lmhead_logps``, a ``torch.autograd.Function`` front
end for training code. ``lmhead_logps`` and ``lmhead_distill`` take the final
norm too (``norm=Norm(...)``: hidden is then the stream in front of it).
"""
from __future__ import annotations

import contextlib
import math
from typing import Any, NamedTuple, Optional, Tuple

from . import _native
from ._native import LmheadError, load, version  # noqa: F401

__all__ = [
    "LmheadError",
    "lmhead_logps_workspace_bytes",
    "lmhead_logps_fwd",
    "lmhead_logps_bwd",
    "lmhead_logps_fwd_temp",
    "lmhead_logps_bwd_temp",
    "lmhead_logps_bwd_ex",
    "lmhead_logps_bwd_bf16",
    "lmhead_logps_fwd_shard",
    "lmhead_logps_merge_shards",
    "lmhead_logps_bwd_shard",
    "lmhead_logps_fwd_noalloc",
    "lmhead_logps_distill_workspace_bytes",
    "lmhead_logps_distill_fwd",
    "lmhead_logps_distill_bwd",
    "lmhead_logps_norm_workspace_bytes",
    "lmhead_logps_norm_fwd",
    "lmhead_logps_norm_bwd",
    "lmhead_logps_embed_workspace_bytes",
    "lmhead_logps_embed_fwd",
    "lmhead_logps_embed_bwd",
    "lmhead_logps_beam_workspace_bytes",
    "lmhead_logps_beam_step",
    "lmhead_logps_beam_reorder",
    "lmhead_logps",
    "lmhead_distill",
    "lmhead_norm",
    "lmhead_embed",
    "Norm",
    "forward",
    "backward",
    "distill_forward",
    "distill_backward",
    "norm_forward",
    "norm_backward",
    "embed_forward",
    "embed_backward",
    "beam_step",
    "beam_reorder",
    "workspace_for",
    "distill_workspace_for",
    "norm_workspace_for",
    "embed_workspace_for",
    "beam_workspace_for",
    "version",
]


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t, name, dtypes, device, numel=None, optional=False):
    # the usual cases first: small calls are bound by what is done here
    if t is None and optional:
        return 0
    try:
        if (t.dtype in dtypes and t.is_cuda and t.device == device and t.is_contiguous()
                and (numel is None or t.numel() == numel)):
            return t.data_ptr()
    except AttributeError:
        pass
    torch = _torch()
    if t is None:
        if optional:
            return 0
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a GPU, got {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


_BF16_TYPES = ()


def _bf16_types():
    global _BF16_TYPES
    if not _BF16_TYPES:
        torch = _torch()
        _BF16_TYPES = (torch.bfloat16, torch.int16, torch.uint16)
    return _BF16_TYPES


def _stream(device, stream):
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # without building a Stream object
        if raw is not None and device.index is not None:
            return raw(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _enqueue(dev, raw, *args):
    """Call ``raw`` with the tensors' device current (a launch goes to the
    current device where the stream is the default one) and check its status."""
    torch = _torch()
    if dev.index is None or dev.index == torch.cuda.current_device():
        _native.check(raw(*args))
    else:
        with torch.cuda.device(dev):
            _native.check(raw(*args))


def _allocating(device, stream):
    """Context in which tensors are allocated for work on ``stream`` (None: the
    current one): from that stream's own pool, so that neither their earlier
    nor their later use elsewhere overlaps it."""
    torch = _torch()
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def lmhead_logps_workspace_bytes(N: int, H: int, V: int, chunk_size: int, with_backward=True) -> int:
    """Workspace bytes: with_backward False (forward only), True (forward and
    the float32-gradient backward) or "bf16" (also the bf16-gradient backward)."""
    return _native.raw_workspace_bytes(N, H, V, chunk_size, _ws_kind(with_backward))


def _ws_kind(with_backward) -> int:
    if with_backward == "bf16":
        return _native.WS_BWD_BF16
    if isinstance(with_backward, str):
        raise ValueError(f"with_backward must be a bool or 'bf16', got {with_backward!r}")
    return _native.WS_BWD if with_backward else _native.WS_FWD


def _shapes(hidden, W, targets):
    if hidden.dim() != 2 or W.dim() != 2 or hidden.shape[1] != W.shape[1]:
        raise ValueError(f"hidden [N,H] and W [V,H] must share H: {tuple(hidden.shape)} vs {tuple(W.shape)}")
    N, H = hidden.shape
    V = W.shape[0]
    if targets.numel() != N:
        raise ValueError(f"targets has {targets.numel()} entries, expected {N}")
    return int(N), int(H), int(V)


def _fwd_args(hidden, W, targets, chunk_size, logp, entropy, lse, workspace, stream):
    torch = _torch()
    N, H, V = _shapes(hidden, W, targets)
    dev = hidden.device
    ptrs = (
        _ptr(hidden, "hidden", _bf16_types(), dev),
        _ptr(W, "W", _bf16_types(), dev),
        _ptr(targets, "targets", (torch.int32,), dev),
        N, H, V, chunk_size,
    )
    outs = (
        _ptr(logp, "logp", (torch.float32,), dev, N),
        _ptr(entropy, "entropy", (torch.float32,), dev, N, optional=True),
        _ptr(lse, "lse", (torch.float32,), dev, N),
        _ptr(workspace, "workspace", (torch.uint8,), dev),
        workspace.numel(),
        _stream(dev, stream),
    )
    return ptrs, outs


def lmhead_logps_fwd(hidden, W, targets, chunk_size: int, logp, entropy, lse, workspace, stream=None) -> None:
    """Enqueue the forward on ``stream`` (default: torch's current stream)."""
    ptrs, outs = _fwd_args(hidden, W, targets, chunk_size, logp, entropy, lse, workspace, stream)
    _enqueue(hidden.device, _native.raw_fwd, *ptrs, *outs)


def lmhead_logps_fwd_temp(hidden, W, targets, chunk_size: int, temperature: float, logp, entropy, lse, workspace,
                          stream=None) -> None:
    """Enqueue the tempered forward (logits / temperature) on ``stream``."""
    ptrs, outs = _fwd_args(hidden, W, targets, chunk_size, logp, entropy, lse, workspace, stream)
    _enqueue(hidden.device, _native.raw_fwd_temp, *ptrs, temperature, *outs)


def lmhead_logps_fwd_noalloc(hidden, W, targets, chunk_size: int, temperature: float, logp, entropy, lse,
                             stream=None) -> None:
    """Enqueue the tempered forward without a workspace (the library's fixed
    scratch array; calls that overlap on one GPU race)."""
    torch = _torch()
    N, H, V = _shapes(hidden, W, targets)
    dev = hidden.device
    _enqueue(
        dev, _native.raw_fwd_noalloc,
        _ptr(hidden, "hidden", _bf16_types(), dev), _ptr(W, "W", _bf16_types(), dev),
        _ptr(targets, "targets", (torch.int32,), dev), N, H, V, chunk_size, temperature,
        _ptr(logp, "logp", (torch.float32,), dev, N), _ptr(entropy, "entropy", (torch.float32,), dev, N, optional=True),
        _ptr(lse, "lse", (torch.float32,), dev, N), _stream(dev, stream))


def _bwd_args(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream,
              grad_types=None):
    torch = _torch()
    if grad_types is None:
        grad_types = (torch.float32,)
    N, H, V = _shapes(hidden, W, targets)
    dev = hidden.device
    if tuple(dh.shape) != (N, H) or tuple(dW.shape) != (V, H):
        raise ValueError("dh must be [N,H] and dW [V,H]")
    ptrs = (
        _ptr(hidden, "hidden", _bf16_types(), dev),
        _ptr(W, "W", _bf16_types(), dev),
        _ptr(targets, "targets", (torch.int32,), dev),
        N, H, V, chunk_size,
    )
    rest = (
        _ptr(lse, "lse", (torch.float32,), dev, N),
        _ptr(entropy, "entropy", (torch.float32,), dev, N, optional=True),
        _ptr(g_logp, "g_logp", (torch.float32,), dev, N, optional=True),
        _ptr(g_ent, "g_ent", (torch.float32,), dev, N, optional=True),
        _ptr(dh, "dh", grad_types, dev),
        _ptr(dW, "dW", grad_types, dev),
        _ptr(workspace, "workspace", (torch.uint8,), dev),
        workspace.numel(),
        _stream(dev, stream),
    )
    return ptrs, rest


def lmhead_logps_bwd(hidden, W, targets, chunk_size: int, lse, entropy, g_logp, g_ent, dh, dW, workspace,
                     stream=None) -> None:
    """Enqueue the backward on ``stream`` (default: torch's current stream)."""
    ptrs, rest = _bwd_args(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream)
    _enqueue(hidden.device, _native.raw_bwd, *ptrs, *rest)


def lmhead_logps_bwd_temp(hidden, W, targets, chunk_size: int, temperature: float, lse, entropy, g_logp, g_ent,
                          dh, dW, workspace, stream=None) -> None:
    """Enqueue the tempered backward on ``stream``; lse and entropy come from
    the tempered forward with the same temperature."""
    ptrs, rest = _bwd_args(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream)
    _enqueue(hidden.device, _native.raw_bwd_temp, *ptrs, temperature, *rest)


def lmhead_logps_bwd_ex(hidden, W, targets, chunk_size: int, temperature: float, lse, entropy, g_logp, g_ent,
                        dh, dW, flags: int, workspace, stream=None) -> None:
    """Enqueue the backward with flags (``_native.BWD_ACCUMULATE_DH`` /
    ``BWD_ACCUMULATE_DW``: add into dh / dW instead of overwriting)."""
    ptrs, rest = _bwd_args(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream)
    _enqueue(hidden.device, _native.raw_bwd_ex, *ptrs, temperature, *rest[:6], flags, *rest[6:])


def lmhead_logps_bwd_bf16(hidden, W, targets, chunk_size: int, temperature: float, lse, entropy, g_logp, g_ent,
                          dh, dW, flags: int, workspace, stream=None) -> None:
    """Enqueue the backward writing bf16 gradients dh [N, H] / dW [V, H]
    (bfloat16 tensors); ``flags`` as for ``lmhead_logps_bwd_ex``; the
    workspace is sized with ``with_backward="bf16"``."""
    ptrs, rest = _bwd_args(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream,
                           grad_types=_bf16_types())
    _enqueue(hidden.device, _native.raw_bwd_bf16, *ptrs, temperature, *rest[:6], flags, *rest[6:])


def lmhead_logps_fwd_shard(hidden, W_shard, targets, vocab_offset: int, V_total: int, chunk_size: int,
                           temperature: float, partial, workspace, stream=None) -> None:
    """Enqueue one vocabulary shard's forward: partial f32 [N, 4] records."""
    torch = _torch()
    N, H, V = _shapes(hidden, W_shard, targets)
    dev = hidden.device
    _enqueue(
        dev, _native.raw_fwd_shard,
        _ptr(hidden, "hidden", _bf16_types(), dev), _ptr(W_shard, "W_shard", _bf16_types(), dev),
        _ptr(targets, "targets", (torch.int32,), dev), N, H, V, vocab_offset, V_total, chunk_size, temperature,
        _ptr(partial, "partial", (torch.float32,), dev, 4 * N), _ptr(workspace, "workspace", (torch.uint8,), dev),
        workspace.numel(), _stream(dev, stream))


def lmhead_logps_merge_shards(partials, targets, V_total: int, temperature: float, logp, entropy, lse,
                              stream=None) -> None:
    """Merge shard records partials f32 [P, N, 4] (shard order) into logp / entropy / lse."""
    torch = _torch()
    if partials.dim() != 3 or partials.shape[2] != 4:
        raise ValueError("partials must be [P, N, 4]")
    P, N = int(partials.shape[0]), int(partials.shape[1])
    dev = partials.device
    _enqueue(
        dev, _native.raw_merge_shards,
        _ptr(partials, "partials", (torch.float32,), dev), P, _ptr(targets, "targets", (torch.int32,), dev, N),
        N, V_total, temperature, _ptr(logp, "logp", (torch.float32,), dev, N),
        _ptr(entropy, "entropy", (torch.float32,), dev, N, optional=True), _ptr(lse, "lse", (torch.float32,), dev, N),
        _stream(dev, stream))


def lmhead_logps_bwd_shard(hidden, W_shard, targets, vocab_offset: int, V_total: int, chunk_size: int,
                           temperature: float, lse, entropy, g_logp, g_ent, dh, dW_shard, flags: int, workspace,
                           stream=None) -> None:
    """Enqueue one vocabulary shard's backward (dW_shard, and its part of dh)."""
    ptrs, rest = _bwd_args(hidden, W_shard, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW_shard,
                           workspace, stream)
    hid, Wp, tg, N, H, V, C = ptrs
    _enqueue(hidden.device, _native.raw_bwd_shard, hid, Wp, tg, N, H, V, vocab_offset, V_total, C, temperature,
             *rest[:6], flags, *rest[6:])


def workspace_for(hidden, W, chunk_size: int, with_backward=True):
    """Allocate a workspace (uint8 tensor) for the given calls: with_backward
    False, True or "bf16" as for ``lmhead_logps_workspace_bytes``."""
    torch = _torch()
    N, H = hidden.shape
    V = W.shape[0]
    nbytes = lmhead_logps_workspace_bytes(N, H, V, chunk_size, with_backward)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=hidden.device)


def forward(hidden, W, targets, chunk_size: int, with_entropy: bool = True, workspace=None,
            stream=None, temperature: Optional[float] = None) -> Tuple:
    """Allocate outputs (torch) and run the forward: (logp, entropy | None, lse).
    ``temperature`` (None: the untempered call) scores the logits divided by it."""
    torch = _torch()
    N = hidden.shape[0]
    dev = hidden.device
    with _allocating(dev, stream):
        logp = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        ent = torch.empty(N, dtype=torch.float32, device=dev) if with_entropy else None
        if workspace is None:
            workspace = workspace_for(hidden, W, chunk_size, with_backward=False)
    if temperature is None:
        lmhead_logps_fwd(hidden, W, targets, chunk_size, logp, ent, lse, workspace, stream)
    else:
        lmhead_logps_fwd_temp(hidden, W, targets, chunk_size, temperature, logp, ent, lse, workspace, stream)
    return logp, ent, lse


def backward(hidden, W, targets, chunk_size: int, lse, entropy, g_logp, g_ent: Optional = None,
             workspace=None, stream=None, temperature: Optional[float] = None, dh=None, dW=None,
             accumulate: bool = False, grad_dtype=None) -> Tuple:
    """Run the backward: (dh, dW), float32 (or bfloat16 with
    ``grad_dtype=torch.bfloat16``). Gradients are allocated unless ``dh`` /
    ``dW`` are given; with ``accumulate`` the given buffers are added into.
    ``temperature`` must match the forward that produced lse and entropy."""
    torch = _torch()
    N, H = hidden.shape
    V = W.shape[0]
    dev = hidden.device
    if grad_dtype is None:
        grad_dtype = dh.dtype if dh is not None else torch.float32
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    if accumulate and (dh is None or dW is None):
        raise ValueError("accumulate needs both dh and dW buffers")
    with _allocating(dev, stream):
        if dh is None:
            dh = torch.empty((N, H), dtype=grad_dtype, device=dev)
        if dW is None:
            dW = torch.empty((V, H), dtype=grad_dtype, device=dev)
        if workspace is None:
            workspace = workspace_for(hidden, W, chunk_size,
                                      with_backward="bf16" if grad_dtype == torch.bfloat16 else True)
    if grad_dtype == torch.bfloat16:
        flags = (_native.BWD_ACCUMULATE_DH | _native.BWD_ACCUMULATE_DW) if accumulate else 0
        lmhead_logps_bwd_bf16(hidden, W, targets, chunk_size, 1.0 if temperature is None else temperature, lse,
                              entropy, g_logp, g_ent, dh, dW, flags, workspace, stream)
        return dh, dW
    if accumulate:
        flags = _native.BWD_ACCUMULATE_DH | _native.BWD_ACCUMULATE_DW
        lmhead_logps_bwd_ex(hidden, W, targets, chunk_size, 1.0 if temperature is None else temperature, lse,
                            entropy, g_logp, g_ent, dh, dW, flags, workspace, stream)
    elif temperature is None:
        lmhead_logps_bwd(hidden, W, targets, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace, stream)
    else:
        lmhead_logps_bwd_temp(hidden, W, targets, chunk_size, temperature, lse, entropy, g_logp, g_ent, dh, dW,
                              workspace, stream)
    return dh, dW


def lmhead_logps_distill_workspace_bytes(N: int, H: int, V: int, K: int, chunk_size: int, with_backward=True) -> int:
    """Workspace bytes of the distillation calls; with_backward as for
    ``lmhead_logps_workspace_bytes``."""
    return _native.raw_distill_workspace_bytes(N, H, V, K, chunk_size, _ws_kind(with_backward))


def _type_of(t, name):
    code = _any_types().get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}, expected float32 or bfloat16")
    return code


_F32_TYPES = ()


def _f32_types():
    global _F32_TYPES
    if not _F32_TYPES:
        _F32_TYPES = (_torch().float32,)
    return _F32_TYPES


_ANY_TYPES = {}


def _any_types():
    """dtype -> type code of what holds float32 or bfloat16 values."""
    if not _ANY_TYPES:
        _ANY_TYPES.update({t: _native.TYPE_BF16 for t in _bf16_types()})
        _ANY_TYPES[_torch().float32] = _native.TYPE_F32
    return _ANY_TYPES


def _distill_args(hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature):
    torch = _torch()
    if hidden.dim() != 2 or W.dim() != 2 or hidden.shape[1] != W.shape[1]:
        raise ValueError(f"hidden [N,H] and W [V,H] must share H: {tuple(hidden.shape)} vs {tuple(W.shape)}")
    N, H = hidden.shape
    V = W.shape[0]
    if ids.dim() != 2 or ids.shape[0] != N or teacher.shape != ids.shape:
        raise ValueError(f"ids and teacher must be [{N}, K]: {tuple(ids.shape)} and {tuple(teacher.shape)}")
    K = ids.shape[1]
    dev = hidden.device
    return dev, N, K, (
        _ptr(hidden, "hidden", _bf16_types(), dev), _ptr(W, "W", _bf16_types(), dev),
        _ptr(targets, "targets", (torch.int32,), dev, N, optional=True), _ptr(ids, "ids", (torch.int32,), dev),
        _ptr(teacher, "teacher", _any_types(), dev), _type_of(teacher, "teacher"),
        _ptr(teacher_lse, "teacher_lse", (torch.float32,), dev, N, optional=True), N, H, V, K, chunk_size, temperature)


def lmhead_logps_distill_fwd(hidden, W, targets, ids, teacher, teacher_lse, chunk_size: int, temperature: float, kl,
                             logp, lse, logp_top, workspace, stream=None) -> None:
    """Enqueue the distillation forward: kl [N], logp [N] (or None), lse [N]
    and logp_top [N, K] (float32). ``targets`` (int32 [N]) and ``teacher_lse``
    (float32 [N]) may be None; ``ids`` is int32 [N, K], ``teacher`` float32 or
    bfloat16 [N, K]."""
    f32 = _f32_types()
    dev, N, K, args = _distill_args(hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature)
    _enqueue(
        dev, _native.raw_distill_fwd, *args, _ptr(kl, "kl", f32, dev, N), _ptr(logp, "logp", f32, dev, N, optional=True), _ptr(lse, "lse", f32, dev, N),
        _ptr(logp_top, "logp_top", f32, dev, N * K), _ptr(workspace, "workspace", (_torch().uint8,), dev),
        workspace.numel(), _stream(dev, stream))


def lmhead_logps_distill_bwd(hidden, W, targets, ids, teacher, teacher_lse, chunk_size: int, temperature: float, logp,
                             lse, logp_top, g_kl, g_logp, dh, dW, flags: int, workspace, stream=None) -> None:
    """Enqueue the distillation backward into dh [N, H] / dW [V, H], both
    float32 or both bfloat16; ``flags`` as for ``lmhead_logps_bwd_ex``; the
    workspace is that of ``distill_workspace_for`` (True or "bf16")."""
    f32 = _f32_types()
    dev, N, K, args = _distill_args(hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature)
    if dh.shape != hidden.shape or dW.shape != W.shape:
        raise ValueError("dh must be [N,H] and dW [V,H]")
    if dh.dtype != dW.dtype:
        raise TypeError(f"dh and dW must have one dtype, got {dh.dtype} and {dW.dtype}")
    _enqueue(
        dev, _native.raw_distill_bwd, *args, _ptr(logp, "logp", f32, dev, N, optional=True), _ptr(lse, "lse", f32, dev, N),
        _ptr(logp_top, "logp_top", f32, dev, N * K), _ptr(g_kl, "g_kl", f32, dev, N, optional=True),
        _ptr(g_logp, "g_logp", f32, dev, N, optional=True), _ptr(dh, "dh", _any_types(), dev),
        _ptr(dW, "dW", _any_types(), dev), _type_of(dh, "dh"), flags,
        _ptr(workspace, "workspace", (_torch().uint8,), dev), workspace.numel(), _stream(dev, stream))


def distill_workspace_for(hidden, W, ids, chunk_size: int, with_backward=True):
    """Allocate a workspace for the distillation calls (with_backward as for
    ``workspace_for``)."""
    torch = _torch()
    nbytes = lmhead_logps_distill_workspace_bytes(hidden.shape[0], hidden.shape[1], W.shape[0], ids.shape[1],
                                                  chunk_size, with_backward)
    return torch.empty(nbytes, dtype=torch.uint8, device=hidden.device)


def distill_forward(hidden, W, targets, ids, teacher, chunk_size: int, teacher_lse=None, workspace=None, stream=None,
                    temperature: float = 1.0) -> Tuple:
    """Allocate outputs and run the distillation forward: (kl, logp | None,
    lse, logp_top); ``targets`` may be None."""
    torch = _torch()
    N, K = ids.shape
    dev = hidden.device
    with _allocating(dev, stream):
        kl, lse = (torch.empty(N, dtype=torch.float32, device=dev) for _ in range(2))
        logp = None if targets is None else torch.empty(N, dtype=torch.float32, device=dev)
        logp_top = torch.empty((N, K), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = distill_workspace_for(hidden, W, ids, chunk_size, with_backward=False)
    lmhead_logps_distill_fwd(hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature, kl, logp, lse,
                             logp_top, workspace, stream)
    return kl, logp, lse, logp_top


def distill_backward(hidden, W, targets, ids, teacher, chunk_size: int, logp, lse, logp_top, g_kl, g_logp=None,
                     teacher_lse=None, workspace=None, stream=None, temperature: float = 1.0, dh=None, dW=None,
                     accumulate: bool = False, grad_dtype=None) -> Tuple:
    """Run the distillation backward: (dh, dW), float32 (or bfloat16 with
    ``grad_dtype=torch.bfloat16``); the rest as for ``backward``."""
    torch = _torch()
    if grad_dtype is None:
        grad_dtype = dh.dtype if dh is not None else torch.float32
    if grad_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    if accumulate and (dh is None or dW is None):
        raise ValueError("accumulate needs both dh and dW buffers")
    with _allocating(hidden.device, stream):
        if dh is None:
            dh = torch.empty(hidden.shape, dtype=grad_dtype, device=hidden.device)
        if dW is None:
            dW = torch.empty(W.shape, dtype=grad_dtype, device=hidden.device)
        if workspace is None:
            workspace = distill_workspace_for(hidden, W, ids, chunk_size,
                                              with_backward="bf16" if grad_dtype == torch.bfloat16 else True)
    flags = (_native.BWD_ACCUMULATE_DH | _native.BWD_ACCUMULATE_DW) if accumulate else 0
    lmhead_logps_distill_bwd(hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature, logp, lse,
                             logp_top, g_kl, g_logp, dh, dW, flags, workspace, stream)
    return dh, dW


class Norm(NamedTuple):
    """A norm over the last dimension: weight and bias [H] (or None), eps, and
    kind "layer" or "rms"."""
    weight: Any = None
    bias: Any = None
    eps: float = 1e-6
    kind: str = "layer"


_NORM_KINDS = {"layer": _native.NORM_LAYER, "rms": _native.NORM_RMS}


def _norm_kind(kind):
    code = _NORM_KINDS.get(kind)
    if code is None:
        raise ValueError(f"kind must be 'layer' or 'rms', got {kind!r}")
    return code


def _norm_shape(x):
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x must have a last dimension to normalise, and it must not be empty")
    return x.numel() // shape[-1], shape[-1]


def lmhead_logps_norm_workspace_bytes(N: int, H: int) -> int:
    """Workspace bytes of the norm's backward."""
    return _native.raw_norm_workspace_bytes(N, H)


def _vector_type(a, b, name_a, name_b):
    """The one type of two optional vectors (float32 if there is neither)."""
    if a is None:
        return _native.TYPE_F32 if b is None else _type_of(b, name_b)
    if b is not None and a.dtype != b.dtype:
        raise TypeError(f"{name_a} and {name_b} must have one dtype, got {a.dtype} and {b.dtype}")
    return _type_of(a, name_a)


def lmhead_logps_norm_fwd(x, weight, bias, eps: float, kind: str, y, mean, rstd, stream=None) -> None:
    """Enqueue the norm of x [..., H] into y (x's shape; bfloat16, or float32
    where x is). weight and bias [H] may be None, and mean / rstd (float32,
    one per row, for the backward) too; kind is "layer" or "rms"."""
    any_, f32 = _any_types(), _f32_types()
    N, H = _norm_shape(x)
    dev = x.device
    if y.shape != x.shape:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected {tuple(x.shape)}")
    _enqueue(
        dev, _native.raw_norm_fwd, _ptr(x, "x", any_, dev), any_[x.dtype],
        _ptr(weight, "weight", any_, dev, H, True), _ptr(bias, "bias", any_, dev, H, True),
        _vector_type(weight, bias, "weight", "bias"), N, H, eps, _norm_kind(kind), _ptr(y, "y", any_, dev),
        any_[y.dtype], _ptr(mean, "mean", f32, dev, N, True), _ptr(rstd, "rstd", f32, dev, N, True),
        _stream(dev, stream))


def lmhead_logps_norm_bwd(x, weight, kind: str, mean, rstd, dy, dx, dweight, dbias, flags: int, workspace,
                          stream=None) -> None:
    """Enqueue the norm's backward into dx (x's dtype) and, unless None,
    dweight and dbias [H] (float32 or bfloat16); ``flags`` 0 or
    ``_native.BWD_ACCUMULATE_DW`` (add into dweight and dbias). The workspace
    may be None where neither is wanted."""
    any_, f32 = _any_types(), _f32_types()
    N, H = _norm_shape(x)
    dev = x.device
    if dy.shape != x.shape or dx.shape != x.shape:
        raise ValueError(f"dy and dx must have x's shape {tuple(x.shape)}, got {tuple(dy.shape)} and {tuple(dx.shape)}")
    x_type = _type_of(x, "x")
    if _type_of(dx, "dx") != x_type:
        raise TypeError(f"dx must have x's dtype {x.dtype}, got {dx.dtype}")
    _enqueue(
        dev, _native.raw_norm_bwd, _ptr(x, "x", any_, dev), x_type, _ptr(weight, "weight", any_, dev, H, True),
        _vector_type(weight, None, "weight", ""), N, H, _norm_kind(kind), _ptr(mean, "mean", f32, dev, N, True),
        _ptr(rstd, "rstd", f32, dev, N), _ptr(dy, "dy", any_, dev), any_[dy.dtype], _ptr(dx, "dx", any_, dev),
        _ptr(dweight, "dweight", any_, dev, H, True), _ptr(dbias, "dbias", any_, dev, H, True),
        _vector_type(dweight, dbias, "dweight", "dbias"), flags,
        _ptr(workspace, "workspace", (_torch().uint8,), dev, None, True), 0 if workspace is None else workspace.numel(),
        _stream(dev, stream))


def norm_workspace_for(x):
    """Allocate a workspace for the norm's backward."""
    torch = _torch()
    N, H = _norm_shape(x)
    return torch.empty(lmhead_logps_norm_workspace_bytes(N, H), dtype=torch.uint8, device=x.device)


def norm_forward(x, weight=None, bias=None, eps: float = 1e-6, kind: str = "layer", out_dtype=None,
                 stream=None) -> Tuple:
    """Allocate outputs and run the norm: (y, mean | None, rstd). ``out_dtype``
    (default: x's) may be bfloat16 for a float32 x."""
    torch = _torch()
    N, _ = _norm_shape(x)
    with _allocating(x.device, stream):
        y = torch.empty(x.shape, dtype=x.dtype if out_dtype is None else out_dtype, device=x.device)
        rstd = torch.empty(N, dtype=torch.float32, device=x.device)
        mean = torch.empty_like(rstd) if kind == "layer" else None
    lmhead_logps_norm_fwd(x, weight, bias, eps, kind, y, mean, rstd, stream)
    return y, mean, rstd


def norm_backward(x, weight, mean, rstd, dy, kind: str = "layer", with_weight: bool = True, with_bias: bool = False,
                  workspace=None, stream=None, dweight=None, dbias=None, accumulate: bool = False,
                  grad_dtype=None) -> Tuple:
    """Run the norm's backward: (dx, dweight | None, dbias | None).
    ``with_weight`` / ``with_bias`` allocate those gradients (in ``grad_dtype``,
    default the weight's dtype or float32) unless buffers are given; with
    ``accumulate`` the given buffers are added into."""
    torch = _torch()
    _, H = _norm_shape(x)
    if accumulate and ((with_weight and dweight is None) or (with_bias and dbias is None)):
        raise ValueError("accumulate needs the gradient buffers that are wanted")
    if grad_dtype is None:
        given = dweight if dweight is not None else dbias if dbias is not None else weight
        grad_dtype = torch.float32 if given is None else given.dtype
    with _allocating(x.device, stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if dweight is None and with_weight:
            dweight = torch.empty(H, dtype=grad_dtype, device=x.device)
        if dbias is None and with_bias:
            dbias = torch.empty(H, dtype=grad_dtype, device=x.device)
        if workspace is None and (dweight is not None or dbias is not None):
            workspace = norm_workspace_for(x)
    flags = _native.BWD_ACCUMULATE_DW if accumulate else 0
    lmhead_logps_norm_bwd(x, weight, kind, mean, rstd, dy, dx, dweight, dbias, flags, workspace, stream)
    return dx, dweight, dbias


def lmhead_logps_embed_workspace_bytes(N: int, H: int, V: int) -> int:
    """Workspace bytes of the embedding's backward."""
    return _native.raw_embed_workspace_bytes(N, H, V)


_I32_TYPES = ()


def _i32_types():
    global _I32_TYPES
    if not _I32_TYPES:
        _I32_TYPES = (_torch().int32,)
    return _I32_TYPES


def _embed_shape(ids, W, y, name):
    if W.dim() != 2:
        raise ValueError(f"the table must be [V, H], got {tuple(W.shape)}")
    V, H = W.shape
    if y.shape != (*ids.shape, H):
        raise ValueError(f"{name} has shape {tuple(y.shape)}, expected {(*ids.shape, H)}")
    return ids.numel(), H, V


def lmhead_logps_embed_fwd(W, ids, scale: float, y, stream=None) -> None:
    """Enqueue the embedding lookup: y [..., H] = scale * W[ids], W [V, H] and
    y float32 or bfloat16 (in any combination), ids int32 [...]. Ids outside
    [0, V) give zeros."""
    any_ = _any_types()
    N, H, V = _embed_shape(ids, W, y, "y")
    dev = W.device
    _enqueue(
        dev, _native.raw_embed_fwd, _ptr(W, "W", any_, dev), any_[W.dtype], _ptr(ids, "ids", _i32_types(), dev), N, H, V,
        scale, _ptr(y, "y", any_, dev), any_[y.dtype], _stream(dev, stream))


def lmhead_logps_embed_bwd(ids, dy, scale: float, dW, flags: int, workspace, stream=None) -> None:
    """Enqueue the embedding's backward into dW [V, H] (float32 or bfloat16):
    ``flags`` 0 writes all of it, ``_native.BWD_ACCUMULATE_DW`` adds into it
    and touches only the rows of words that occur (a tied table, whose head's
    backward wrote dW before). dy is [..., H]; the workspace is that of
    ``embed_workspace_for``."""
    any_ = _any_types()
    N, H, V = _embed_shape(ids, dW, dy, "dy")
    dev = dW.device
    _enqueue(
        dev, _native.raw_embed_bwd, _ptr(ids, "ids", _i32_types(), dev), _ptr(dy, "dy", any_, dev), any_[dy.dtype], N, H, V,
        scale, _ptr(dW, "dW", any_, dev), any_[dW.dtype], flags, _ptr(workspace, "workspace", (_torch().uint8,), dev),
        workspace.numel(), _stream(dev, stream))


def embed_workspace_for(ids, W):
    """Allocate a workspace for the embedding's backward (W: the table or its
    gradient)."""
    torch = _torch()
    V, H = W.shape
    return torch.empty(lmhead_logps_embed_workspace_bytes(ids.numel(), H, V), dtype=torch.uint8, device=W.device)


def embed_forward(W, ids, scale: float = 1.0, out_dtype=None, stream=None):
    """Allocate y [..., H] (in ``out_dtype``, default W's) and run the lookup."""
    torch = _torch()
    with _allocating(W.device, stream):
        y = torch.empty((*ids.shape, W.shape[1]), dtype=W.dtype if out_dtype is None else out_dtype, device=W.device)
    lmhead_logps_embed_fwd(W, ids, scale, y, stream)
    return y


def embed_backward(ids, dy, vocab: Optional[int] = None, scale: float = 1.0, workspace=None, stream=None, dW=None,
                   accumulate: bool = False, grad_dtype=None):
    """Run the embedding's backward: dW [vocab, H], allocated in
    ``grad_dtype`` (default float32) unless given; with ``accumulate`` the
    given buffer is added into."""
    torch = _torch()
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs the dW buffer")
        if vocab is None:
            raise ValueError("vocab (the table's rows) or dW is needed")
    with _allocating(dy.device, stream):
        if dW is None:
            dW = torch.empty((vocab, dy.shape[-1]), dtype=torch.float32 if grad_dtype is None else grad_dtype,
                             device=dy.device)
        if workspace is None:
            workspace = embed_workspace_for(ids, dW)
    lmhead_logps_embed_bwd(ids, dy, scale, dW, _native.BWD_ACCUMULATE_DW if accumulate else 0, workspace, stream)
    return dW


def lmhead_logps_beam_workspace_bytes(N: int, H: int, V: int, beams: int, candidates: int) -> int:
    """Workspace bytes of a beam step."""
    return _native.raw_beam_workspace_bytes(N, H, V, beams, candidates)


def lmhead_logps_beam_step(hidden, W, scores, ended, allowed, beams: int, temperature: float, top_scores, top_ids,
                           top_parents, lse, workspace, stream=None) -> None:
    """Enqueue one step of beam search over the rows of hidden [N, H], in
    groups of ``beams`` rows: the best candidates' scores (float32), words and
    parent rows (int32), each [N / beams, candidates], and lse [N]. ``scores``
    is float32 [N]; ``ended`` (int32 [N]: a row with an id in [0, V) has that
    id, at its unchanged score, as its only candidate) and ``allowed`` (int32
    [N, ceil(V / 32)]: the bits of the words that a row may take) may be None."""
    f32, i32 = _f32_types(), _i32_types()
    if hidden.dim() != 2 or W.dim() != 2 or hidden.shape[1] != W.shape[1]:
        raise ValueError(f"hidden [N,H] and W [V,H] must share H: {tuple(hidden.shape)} vs {tuple(W.shape)}")
    N, H = hidden.shape
    V = W.shape[0]
    if top_scores.dim() != 2 or beams < 1 or top_scores.shape[0] * beams != N:
        raise ValueError(f"top_scores must be [N / beams, candidates] with N = {N} and beams = {beams}, got "
                         f"{tuple(top_scores.shape)}")
    groups, C = top_scores.shape
    dev = hidden.device
    _enqueue(
        dev, _native.raw_beam_step, _ptr(hidden, "hidden", _bf16_types(), dev), _ptr(W, "W", _bf16_types(), dev),
        _ptr(scores, "scores", f32, dev, N), _ptr(ended, "ended", i32, dev, N, True),
        _ptr(allowed, "allowed", i32, dev, N * ((V + 31) // 32), True), N, H, V, beams, C, temperature,
        _ptr(top_scores, "top_scores", f32, dev), _ptr(top_ids, "top_ids", i32, dev, groups * C),
        _ptr(top_parents, "top_parents", i32, dev, groups * C), _ptr(lse, "lse", f32, dev, N),
        _ptr(workspace, "workspace", (_torch().uint8,), dev), workspace.numel(), _stream(dev, stream))


def beam_workspace_for(hidden, W, beams: int, candidates: int):
    """Allocate a workspace for beam steps of this shape."""
    torch = _torch()
    nbytes = lmhead_logps_beam_workspace_bytes(hidden.shape[0], hidden.shape[1], W.shape[0], beams, candidates)
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=hidden.device)


def beam_step(hidden, W, scores, beams: int, candidates: Optional[int] = None, ended=None, allowed=None,
              temperature: float = 1.0, norm: Optional["Norm"] = None, workspace=None, stream=None) -> Tuple:
    """Allocate outputs and run one step of beam search: (top_scores, top_ids,
    top_parents, lse), the first three [N / beams, candidates]. ``candidates``
    defaults to 2 * beams, which holds ``beams`` that have not just ended; it is at
    most 64, so groups of more than 32 beams have to name it. With ``norm``, hidden
    is the stream in front of the final norm (bfloat16 or float32)."""
    torch = _torch()
    N, dev = hidden.shape[0], hidden.device
    if candidates is None:
        candidates = 2 * beams
    if beams < 1 or N % beams:
        raise ValueError(f"hidden has {N} rows, which are no groups of {beams} beams")
    if norm is not None:
        hidden, _, _ = norm_forward(hidden, norm.weight, norm.bias, norm.eps, norm.kind, torch.bfloat16, stream)
    with _allocating(dev, stream):
        top_scores = torch.empty((N // beams, candidates), dtype=torch.float32, device=dev)
        top_ids, top_parents = (torch.empty((N // beams, candidates), dtype=torch.int32, device=dev) for _ in range(2))
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = beam_workspace_for(hidden, W, beams, candidates)
    lmhead_logps_beam_step(hidden, W, scores, ended, allowed, beams, temperature, top_scores, top_ids, top_parents, lse,
                           workspace, stream)
    return top_scores, top_ids, top_parents, lse


def lmhead_logps_beam_reorder(states, parents, beams: int, out, lengths=None, row_dim: int = 0,
                              length_dim: Optional[int] = None, stream=None) -> None:
    """Enqueue the reordering of beams' states, of any dtype, whose dimension
    ``row_dim`` holds the N rows: row j of ``out`` (``states`` itself, or a
    tensor like it) takes over row parents[j] (int32 [N]; one outside j's group
    of ``beams`` rows leaves row j as it is). With ``lengths`` (int32 [N], by
    row of states) only the first lengths[parents[j]] steps of dimension
    ``length_dim`` (default: the one after ``row_dim``) are, and the rest of out
    stays."""
    dims = states.dim()
    if dims == 0 or not -dims <= row_dim < dims:
        raise ValueError(f"row_dim {row_dim} is no dimension of states {tuple(states.shape)}")
    row_dim %= dims
    shape = states.shape
    if out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if out.dtype != states.dtype:
        raise TypeError(f"out must have states' dtype {states.dtype}, got {out.dtype}")
    if lengths is None:
        if length_dim is not None:
            raise ValueError("length_dim is given without lengths")
        runs = steps = 1
        step_bytes = math.prod(shape[row_dim + 1:]) * states.element_size()
    else:
        length_dim = row_dim + 1 if length_dim is None else length_dim + dims if length_dim < 0 else length_dim
        if not row_dim < length_dim < dims:
            raise ValueError(f"lengths need a dimension of states {tuple(shape)} after row_dim {row_dim}, got {length_dim}")
        runs, steps = math.prod(shape[row_dim + 1:length_dim]), shape[length_dim]
        step_bytes = math.prod(shape[length_dim + 1:]) * states.element_size()
    N, dev, types, i32 = shape[row_dim], states.device, (states.dtype,), _i32_types()
    _enqueue(
        dev, _native.raw_beam_reorder, _ptr(states, "states", types, dev), _ptr(out, "out", types, dev),
        _ptr(parents, "parents", i32, dev, N), _ptr(lengths, "lengths", i32, dev, N, True), math.prod(shape[:row_dim]), N,
        beams, runs, steps, step_bytes, _stream(dev, stream))


def beam_reorder(states, parents, beams: int, out=None, lengths=None, row_dim: int = 0,
                 length_dim: Optional[int] = None, stream=None):
    """Reorder beams' states in place, or into ``out``; returns the reordered
    tensor."""
    out = states if out is None else out
    lmhead_logps_beam_reorder(states, parents, beams, out, lengths, row_dim, length_dim, stream)
    return out


_ONCE_FN = None


def _once(*grads):
    """What a front end's backward returns: the library's gradients carry no
    graph, so where one is being recorded (create_graph) they are joined to a
    node that refuses a second backward. As constants they would leave a loss
    on them (a gradient penalty) without its gradient, and say nothing."""
    torch = _torch()
    if not torch.is_grad_enabled():
        return grads
    global _ONCE_FN
    if _ONCE_FN is None:
        class _Once(torch.autograd.Function):
            @staticmethod
            def forward(ctx, joined, grad):
                return grad.detach()

            @staticmethod
            def backward(ctx, g):
                raise RuntimeError("the gradients of lmhead_logps, lmhead_distill, lmhead_norm and lmhead_embed take no second backward")

        _ONCE_FN = _Once
    joined = torch.empty(0, requires_grad=True)
    return tuple(None if g is None else _ONCE_FN.apply(joined, g) for g in grads)


def _autograd_function():
    torch = _torch()

    class _LmheadLogps(torch.autograd.Function):
        """logp (and entropy) of the head with its backward through the
        library. The forward holds only its own small workspace (the split
        records) and keeps lse (and entropy) for the backward; the backward
        sizes its workspace when it runs and writes the gradients in the
        inputs' dtype directly (bf16 inputs: lmhead_logps_bwd_bf16, float32
        sums in the workspace, no float32 [N, H] / [V, H] gradient tensors
        and no cast)."""

        @staticmethod
        def forward(ctx, hidden, W, targets, chunk_size, temperature, with_entropy):
            logp, ent, lse = forward(hidden, W, targets, chunk_size, with_entropy=with_entropy,
                                     temperature=temperature)
            ctx.chunk_size = chunk_size
            ctx.temperature = temperature
            ctx.with_entropy = with_entropy
            saved = (hidden, W, targets, lse) + ((ent,) if with_entropy else ())
            ctx.save_for_backward(*saved)
            if with_entropy:
                return logp, ent
            return logp

        @staticmethod
        def backward(ctx, g_logp, g_ent=None):
            hidden, W, targets, lse = ctx.saved_tensors[:4]
            ent = ctx.saved_tensors[4] if ctx.with_entropy else None
            gl = None if g_logp is None else g_logp.detach().contiguous().float()
            ge = None if (g_ent is None or ent is None) else g_ent.detach().contiguous().float()
            bf16 = hidden.dtype == torch.bfloat16 and W.dtype == torch.bfloat16
            dh, dW = backward(hidden, W, targets, ctx.chunk_size, lse, ent if ge is not None else None, gl, ge,
                              temperature=ctx.temperature,
                              grad_dtype=torch.bfloat16 if bf16 else torch.float32)
            return _once(dh.to(hidden.dtype) if ctx.needs_input_grad[0] else None,
                         dW.to(W.dtype) if ctx.needs_input_grad[1] else None,
                         None, None, None, None)

    return _LmheadLogps


def _distill_function():
    torch = _torch()

    class _LmheadDistill(torch.autograd.Function):
        """kl (and logp) of the head with its backward through the library;
        keeps lse, logp and the student's log-probs at the teacher's ids."""

        @staticmethod
        def forward(ctx, hidden, W, targets, ids, teacher, teacher_lse, chunk_size, temperature):
            kl, logp, lse, logp_top = distill_forward(hidden, W, targets, ids, teacher, chunk_size, teacher_lse,
                                                      temperature=temperature)
            ctx.chunk_size = chunk_size
            ctx.temperature = temperature
            ctx.save_for_backward(hidden, W, targets, ids, teacher, teacher_lse, logp, lse, logp_top)
            return kl if logp is None else (kl, logp)

        @staticmethod
        def backward(ctx, g_kl, g_logp=None):
            hidden, W, targets, ids, teacher, teacher_lse, logp, lse, logp_top = ctx.saved_tensors
            gk = None if g_kl is None else g_kl.detach().contiguous().float()
            gl = None if (g_logp is None or logp is None) else g_logp.detach().contiguous().float()
            bf16 = hidden.dtype == torch.bfloat16 and W.dtype == torch.bfloat16
            dh, dW = distill_backward(hidden, W, targets, ids, teacher, ctx.chunk_size, logp, lse, logp_top, gk, gl,
                                      teacher_lse, temperature=ctx.temperature,
                                      grad_dtype=torch.bfloat16 if bf16 else torch.float32)
            return _once(dh.to(hidden.dtype) if ctx.needs_input_grad[0] else None,
                         dW.to(W.dtype) if ctx.needs_input_grad[1] else None,
                         None, None, None, None, None, None)

    return _LmheadDistill


def _norm_function():
    torch = _torch()

    class _LmheadNorm(torch.autograd.Function):
        """The norm with its backward through the library; keeps x and the
        rows' statistics."""

        @staticmethod
        def forward(ctx, x, weight, bias, eps, kind, out_dtype):
            y, mean, rstd = norm_forward(x, weight, bias, eps, kind, out_dtype)
            ctx.kind = kind
            ctx.bias = None if bias is None else bias.dtype
            ctx.save_for_backward(x, weight, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, weight, mean, rstd = ctx.saved_tensors
            want_w, want_b = ctx.needs_input_grad[1], ctx.needs_input_grad[2]
            dx, dw, db = norm_backward(x, weight, mean, rstd, dy.detach().contiguous(), ctx.kind, with_weight=want_w,
                                       with_bias=want_b, grad_dtype=ctx.bias if weight is None else weight.dtype)
            return _once(dx if ctx.needs_input_grad[0] else None, dw, db, None, None, None)

    return _LmheadNorm


def _embed_function():
    torch = _torch()

    class _LmheadEmbed(torch.autograd.Function):
        """The embedding lookup with its backward through the library; keeps
        the ids."""

        @staticmethod
        def forward(ctx, W, ids, scale, out_dtype):
            ctx.scale, ctx.vocab, ctx.dtype = scale, W.shape[0], W.dtype
            ctx.save_for_backward(ids)
            return embed_forward(W, ids, scale, out_dtype)

        @staticmethod
        def backward(ctx, dy):
            ids, = ctx.saved_tensors
            dW = None
            if ctx.needs_input_grad[0]:
                dW = embed_backward(ids, dy.detach().contiguous(), ctx.vocab, ctx.scale, grad_dtype=ctx.dtype)
            return _once(dW, None, None, None)

    return _LmheadEmbed


_FN = None
_DISTILL_FN = None
_NORM_FN = None
_EMBED_FN = None


def lmhead_embed(W, ids, scale: float = 1.0, out_dtype=None):
    """Differentiable embedding lookup: ``scale * W[ids]`` [..., H] in
    ``out_dtype`` (default W's; float32 for a float32 stream), for W [V, H]
    float32 or bfloat16 and ids int32 [...] of any shape; ids outside [0, V) give
    zeros and no gradient. W's gradient comes whole, in W's dtype (a trainer that
    keeps a tied table's gradient in a buffer of its own adds to the rows that
    occur alone with ``embed_backward(..., dW=buffer, accumulate=True)``). The
    backward takes up to 2^23 - 256 ids and words. A second backward, through the
    gradients, is refused."""
    global _EMBED_FN
    if _EMBED_FN is None:
        _EMBED_FN = _embed_function()
    return _EMBED_FN.apply(W, ids, scale, out_dtype)


def lmhead_norm(x, weight=None, bias=None, eps: float = 1e-6, kind: str = "layer", out_dtype=None):
    """Differentiable norm in front of the head: x [..., H] bfloat16 or
    float32 (``out_dtype=torch.bfloat16`` gives the head its dtype from a
    float32 stream); gradients flow to x, weight and bias. A row whose incoming
    gradient is 0 (a token that the head masks) adds nothing to any gradient,
    whatever it holds. A second backward, through the gradients, is refused."""
    global _NORM_FN
    if _NORM_FN is None:
        _NORM_FN = _norm_function()
    return _NORM_FN.apply(x, weight, bias, eps, kind, out_dtype)


def _normed(hidden, norm):
    if norm is None:
        return hidden
    return lmhead_norm(hidden, norm.weight, norm.bias, norm.eps, norm.kind, out_dtype=_torch().bfloat16)


def lmhead_logps(hidden, W, targets, chunk_size: int, temperature: Optional[float] = None, with_entropy: bool = True,
                 norm: Optional[Norm] = None):
    """Differentiable head for training code: returns ``(logp, entropy)``
    (or ``logp`` alone without entropy). ``hidden`` [N, H] and ``W`` [V, H]
    are bfloat16 tensors on one GPU; a backward through either output runs
    ``lmhead_logps_bwd`` on the saved lse / entropy (the logits are recomputed,
    never stored). Masked targets (outside [0, V)) give zeros. With ``norm``,
    hidden is the stream in front of the final norm (bfloat16 or float32), and
    gradients flow to it and to the norm's weight and bias. A second backward,
    through the gradients, is refused."""
    global _FN
    if _FN is None:
        _FN = _autograd_function()
    return _FN.apply(_normed(hidden, norm), W, targets, chunk_size, temperature, with_entropy)


def lmhead_distill(hidden, W, ids, teacher, chunk_size: int, targets=None, teacher_lse=None,
                   temperature: float = 1.0, norm: Optional[Norm] = None):
    """Differentiable distillation loss per token against a teacher's top
    logits: ``kl`` [N], or ``(kl, logp)`` with hard ``targets``. ``ids`` (int32)
    and ``teacher`` (bfloat16 or float32) are [N, K]; ids outside [0, V) are
    missing entries. Gradients flow to hidden and W (and, with ``norm`` as for
    ``lmhead_logps``, to the norm's weight and bias); the teacher gets none.
    Multiply kl by temperature squared for gradients of temperature 1's size.
    ``chunk_size`` bounds the backward's cotangent block as for the head, but
    blocks of up to 2^25 entries (134 MB) are always taken. A backward pass may
    be captured into a graph where no eager graph of the same leaves is alive
    (torch ends the process otherwise, whatever the function). A second backward,
    through the gradients, is refused."""
    global _DISTILL_FN
    if _DISTILL_FN is None:
        _DISTILL_FN = _distill_function()
    return _DISTILL_FN.apply(_normed(hidden, norm), W, targets, ids, teacher, teacher_lse, chunk_size, temperature)
