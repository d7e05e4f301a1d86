"""ctypes binding of the C ABI in ``include/lmhead_logps.h``.

Argument marshalling only: every step of the head runs in the HIP library.
There is no CPU fallback; loading fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
# LMHEAD_LOGPS_LIB names another build of the library to load (the host
# sanitizer build of cross_entropy_amd/build.py --sanitize)
LIB_PATH = os.environ.get("LMHEAD_LOGPS_LIB") or os.path.join(_PKG, "liblmhead_logps.so")

LMH_OK = 0
ERROR_NAMES = {
    -1: "LMH_ERR_NULL",
    -2: "LMH_ERR_SHAPE",
    -3: "LMH_ERR_CHUNK",
    -4: "LMH_ERR_WORKSPACE",
    -5: "LMH_ERR_ARGS",
    -6: "LMH_ERR_UNSUPPORTED",
    -7: "LMH_ERR_HIP",
}

EXPORTED = (
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
    "lmhead_logps_last_error",
    "lmhead_logps_version",
    "lmhead_logps_trace_enable",
    "lmhead_logps_trace_read",
    "lmhead_logps_trace_kernel_name",
)


class LmheadError(RuntimeError):
    """A non-zero status from the library, with its name and message."""

    def __init__(self, code: int, message: str):
        self.code = code
        self.name = ERROR_NAMES.get(code, str(code))
        super().__init__(f"{self.name} ({code}): {message}")


_lib = None


def _hip_runtimes_mapped():
    try:
        with open("/proc/self/maps") as f:
            return sorted({l.split()[-1] for l in f if "libamdhip64" in l})
    except OSError:  # pragma: no cover
        return []


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load (once) and return the HIP library; raise if it is not built.

    PyTorch is imported first so that the library binds to the HIP runtime
    PyTorch already loaded (its wheel bundles one with the same soname):
    device pointers and streams handed over from torch are only valid in
    that runtime. A process that ends up with two HIP runtimes is refused."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: the HIP library is not built "
            "(run `python -m cross_entropy_amd.build` or __graft_entry__.build())")
    import torch  # noqa: F401  (binds the library to torch's HIP runtime)
    lib = ctypes.CDLL(path)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise ImportError(f"two HIP runtimes are loaded in this process: {runtimes}")
    i64, p, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    lib.lmhead_logps_workspace_bytes.argtypes = [i64, i64, i64, i64, ctypes.c_int, ctypes.POINTER(sz)]
    lib.lmhead_logps_workspace_bytes.restype = ctypes.c_int
    lib.lmhead_logps_fwd.argtypes = [p, p, p, i64, i64, i64, i64, p, p, p, p, sz, p]
    lib.lmhead_logps_fwd.restype = ctypes.c_int
    lib.lmhead_logps_bwd.argtypes = [p, p, p, i64, i64, i64, i64, p, p, p, p, p, p, p, sz, p]
    lib.lmhead_logps_bwd.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.lmhead_logps_fwd_temp.argtypes = [p, p, p, i64, i64, i64, i64, f32, p, p, p, p, sz, p]
    lib.lmhead_logps_fwd_temp.restype = ctypes.c_int
    lib.lmhead_logps_bwd_temp.argtypes = [p, p, p, i64, i64, i64, i64, f32, p, p, p, p, p, p, p, sz, p]
    lib.lmhead_logps_bwd_temp.restype = ctypes.c_int
    lib.lmhead_logps_bwd_ex.argtypes = [p, p, p, i64, i64, i64, i64, f32, p, p, p, p, p, p, ctypes.c_uint, p, sz, p]
    lib.lmhead_logps_bwd_ex.restype = ctypes.c_int
    lib.lmhead_logps_bwd_bf16.argtypes = [p, p, p, i64, i64, i64, i64, f32, p, p, p, p, p, p, ctypes.c_uint, p, sz,
                                          p]
    lib.lmhead_logps_bwd_bf16.restype = ctypes.c_int
    lib.lmhead_logps_fwd_shard.argtypes = [p, p, p, i64, i64, i64, i64, i64, i64, f32, p, p, sz, p]
    lib.lmhead_logps_fwd_shard.restype = ctypes.c_int
    lib.lmhead_logps_merge_shards.argtypes = [p, i64, p, i64, i64, f32, p, p, p, p]
    lib.lmhead_logps_merge_shards.restype = ctypes.c_int
    lib.lmhead_logps_bwd_shard.argtypes = [p, p, p, i64, i64, i64, i64, i64, i64, f32, p, p, p, p, p, p,
                                           ctypes.c_uint, p, sz, p]
    lib.lmhead_logps_bwd_shard.restype = ctypes.c_int
    lib.lmhead_logps_fwd_noalloc.argtypes = [p, p, p, i64, i64, i64, i64, f32, p, p, p, p]
    lib.lmhead_logps_fwd_noalloc.restype = ctypes.c_int
    i32 = ctypes.c_int
    lib.lmhead_logps_distill_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32, ctypes.POINTER(sz)]
    lib.lmhead_logps_distill_workspace_bytes.restype = ctypes.c_int
    lib.lmhead_logps_distill_fwd.argtypes = [p, p, p, p, p, i32, p, i64, i64, i64, i64, i64, f32, p, p, p, p, p, sz, p]
    lib.lmhead_logps_distill_fwd.restype = ctypes.c_int
    lib.lmhead_logps_distill_bwd.argtypes = [p, p, p, p, p, i32, p, i64, i64, i64, i64, i64, f32, p, p, p, p, p, p, p,
                                             i32, ctypes.c_uint, p, sz, p]
    lib.lmhead_logps_distill_bwd.restype = ctypes.c_int
    lib.lmhead_logps_norm_workspace_bytes.argtypes = [i64, i64, ctypes.POINTER(sz)]
    lib.lmhead_logps_norm_workspace_bytes.restype = ctypes.c_int
    lib.lmhead_logps_norm_fwd.argtypes = [p, i32, p, p, i32, i64, i64, f32, i32, p, i32, p, p, p]
    lib.lmhead_logps_norm_fwd.restype = ctypes.c_int
    lib.lmhead_logps_norm_bwd.argtypes = [p, i32, p, i32, i64, i64, i32, p, p, p, i32, p, p, p, i32, ctypes.c_uint, p,
                                          sz, p]
    lib.lmhead_logps_norm_bwd.restype = ctypes.c_int
    lib.lmhead_logps_embed_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
    lib.lmhead_logps_embed_workspace_bytes.restype = ctypes.c_int
    lib.lmhead_logps_embed_fwd.argtypes = [p, i32, p, i64, i64, i64, f32, p, i32, p]
    lib.lmhead_logps_embed_fwd.restype = ctypes.c_int
    lib.lmhead_logps_embed_bwd.argtypes = [p, p, i32, i64, i64, i64, f32, p, i32, ctypes.c_uint, p, sz, p]
    lib.lmhead_logps_embed_bwd.restype = ctypes.c_int
    lib.lmhead_logps_beam_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, ctypes.POINTER(sz)]
    lib.lmhead_logps_beam_workspace_bytes.restype = ctypes.c_int
    lib.lmhead_logps_beam_step.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i64, f32, p, p, p, p, p, sz, p]
    lib.lmhead_logps_beam_step.restype = ctypes.c_int
    lib.lmhead_logps_beam_reorder.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, p]
    lib.lmhead_logps_beam_reorder.restype = ctypes.c_int
    lib.lmhead_logps_last_error.argtypes = []
    lib.lmhead_logps_last_error.restype = ctypes.c_char_p
    lib.lmhead_logps_version.argtypes = []
    lib.lmhead_logps_version.restype = ctypes.c_char_p
    lib.lmhead_logps_trace_enable.argtypes = [ctypes.c_int]
    lib.lmhead_logps_trace_enable.restype = ctypes.c_int
    dp = ctypes.POINTER(ctypes.c_double)
    lib.lmhead_logps_trace_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int64), dp, dp, dp]
    lib.lmhead_logps_trace_read.restype = ctypes.c_int
    lib.lmhead_logps_trace_kernel_name.argtypes = [ctypes.c_int]
    lib.lmhead_logps_trace_kernel_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def check(code: int) -> None:
    if code != LMH_OK:
        msg = load().lmhead_logps_last_error().decode(errors="replace")
        raise LmheadError(code, msg)


WS_FWD, WS_BWD, WS_BWD_BF16 = 0, 1, 2


def raw_workspace_bytes(N: int, H: int, V: int, chunk_size: int, with_backward) -> int:
    """with_backward: False / True (WS_FWD / WS_BWD) or WS_BWD_BF16."""
    out = ctypes.c_size_t(0)
    check(load().lmhead_logps_workspace_bytes(int(N), int(H), int(V), int(chunk_size), int(with_backward),
                                              ctypes.byref(out)))
    return int(out.value)


def raw_fwd(hidden, W, targets, N, H, V, chunk_size, logp, entropy, lse, workspace, workspace_bytes,
            stream) -> int:
    """Call lmhead_logps_fwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_fwd(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                   int(chunk_size), logp or None, entropy or None, lse or None,
                                   workspace or None, int(workspace_bytes), stream or None)


def raw_bwd(hidden, W, targets, N, H, V, chunk_size, lse, entropy, g_logp, g_ent, dh, dW, workspace,
            workspace_bytes, stream) -> int:
    """Call lmhead_logps_bwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_bwd(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                   int(chunk_size), lse or None, entropy or None, g_logp or None,
                                   g_ent or None, dh or None, dW or None, workspace or None,
                                   int(workspace_bytes), stream or None)


def raw_fwd_temp(hidden, W, targets, N, H, V, chunk_size, temperature, logp, entropy, lse, workspace,
                 workspace_bytes, stream) -> int:
    """Call lmhead_logps_fwd_temp with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_fwd_temp(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                        int(chunk_size), float(temperature), logp or None, entropy or None,
                                        lse or None, workspace or None, int(workspace_bytes), stream or None)


def raw_bwd_temp(hidden, W, targets, N, H, V, chunk_size, temperature, lse, entropy, g_logp, g_ent, dh, dW,
                 workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_bwd_temp with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_bwd_temp(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                        int(chunk_size), float(temperature), lse or None, entropy or None,
                                        g_logp or None, g_ent or None, dh or None, dW or None,
                                        workspace or None, int(workspace_bytes), stream or None)


BWD_ACCUMULATE_DH = 1
BWD_ACCUMULATE_DW = 2


def raw_bwd_ex(hidden, W, targets, N, H, V, chunk_size, temperature, lse, entropy, g_logp, g_ent, dh, dW, flags,
               workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_bwd_ex with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_bwd_ex(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                      int(chunk_size), float(temperature), lse or None, entropy or None,
                                      g_logp or None, g_ent or None, dh or None, dW or None, int(flags),
                                      workspace or None, int(workspace_bytes), stream or None)


def raw_bwd_bf16(hidden, W, targets, N, H, V, chunk_size, temperature, lse, entropy, g_logp, g_ent, dh, dW, flags,
                 workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_bwd_bf16 with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_bwd_bf16(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                        int(chunk_size), float(temperature), lse or None, entropy or None,
                                        g_logp or None, g_ent or None, dh or None, dW or None, int(flags),
                                        workspace or None, int(workspace_bytes), stream or None)


def raw_fwd_shard(hidden, W_shard, targets, N, H, V_shard, vocab_offset, V_total, chunk_size, temperature,
                  partial, workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_fwd_shard with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_fwd_shard(hidden or None, W_shard or None, targets or None, int(N), int(H),
                                         int(V_shard), int(vocab_offset), int(V_total), int(chunk_size),
                                         float(temperature), partial or None, workspace or None,
                                         int(workspace_bytes), stream or None)


def raw_merge_shards(partials, P, targets, N, V_total, temperature, logp, entropy, lse, stream) -> int:
    """Call lmhead_logps_merge_shards with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_merge_shards(partials or None, int(P), targets or None, int(N), int(V_total),
                                            float(temperature), logp or None, entropy or None, lse or None,
                                            stream or None)


def raw_bwd_shard(hidden, W_shard, targets, N, H, V_shard, vocab_offset, V_total, chunk_size, temperature, lse,
                  entropy, g_logp, g_ent, dh, dW_shard, flags, workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_bwd_shard with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_bwd_shard(hidden or None, W_shard or None, targets or None, int(N), int(H),
                                         int(V_shard), int(vocab_offset), int(V_total), int(chunk_size),
                                         float(temperature), lse or None, entropy or None, g_logp or None,
                                         g_ent or None, dh or None, dW_shard or None, int(flags),
                                         workspace or None, int(workspace_bytes), stream or None)


NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def raw_fwd_noalloc(hidden, W, targets, N, H, V, chunk_size, temperature, logp, entropy, lse, stream) -> int:
    """Call lmhead_logps_fwd_noalloc with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_fwd_noalloc(hidden or None, W or None, targets or None, int(N), int(H), int(V),
                                           int(chunk_size), float(temperature), logp or None, entropy or None,
                                           lse or None, stream or None)


TYPE_BF16, TYPE_F32 = 0, 1
DISTILL_MAX_K = 1024


def raw_distill_workspace_bytes(N: int, H: int, V: int, K: int, chunk_size: int, with_backward) -> int:
    """with_backward: WS_FWD, WS_BWD or WS_BWD_BF16."""
    out = ctypes.c_size_t(0)
    check(load().lmhead_logps_distill_workspace_bytes(int(N), int(H), int(V), int(K), int(chunk_size),
                                                      int(with_backward), ctypes.byref(out)))
    return int(out.value)


def raw_distill_fwd(hidden, W, targets, ids, teacher, teacher_type, teacher_lse, N, H, V, K, chunk_size, temperature,
                    kl, logp, lse, logp_top, workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_distill_fwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_distill_fwd(hidden or None, W or None, targets or None, ids or None, teacher or None,
                                           int(teacher_type), teacher_lse or None, int(N), int(H), int(V), int(K),
                                           int(chunk_size), float(temperature), kl or None, logp or None, lse or None,
                                           logp_top or None, workspace or None, int(workspace_bytes), stream or None)


def raw_distill_bwd(hidden, W, targets, ids, teacher, teacher_type, teacher_lse, N, H, V, K, chunk_size, temperature,
                    logp, lse, logp_top, g_kl, g_logp, dh, dW, grad_type, flags, workspace, workspace_bytes,
                    stream) -> int:
    """Call lmhead_logps_distill_bwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_distill_bwd(hidden or None, W or None, targets or None, ids or None, teacher or None,
                                           int(teacher_type), teacher_lse or None, int(N), int(H), int(V), int(K),
                                           int(chunk_size), float(temperature), logp or None, lse or None,
                                           logp_top or None, g_kl or None, g_logp or None, dh or None, dW or None,
                                           int(grad_type), int(flags), workspace or None, int(workspace_bytes),
                                           stream or None)


NORM_LAYER, NORM_RMS = 0, 1
NORM_MAX_H = 16384


def raw_norm_workspace_bytes(N: int, H: int) -> int:
    out = ctypes.c_size_t(0)
    check(load().lmhead_logps_norm_workspace_bytes(int(N), int(H), ctypes.byref(out)))
    return int(out.value)


def raw_norm_fwd(x, x_type, weight, bias, w_type, N, H, eps, kind, y, y_type, mean, rstd, stream) -> int:
    """Call lmhead_logps_norm_fwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_norm_fwd(x or None, int(x_type), weight or None, bias or None, int(w_type), int(N),
                                        int(H), float(eps), int(kind), y or None, int(y_type), mean or None,
                                        rstd or None, stream or None)


def raw_norm_bwd(x, x_type, weight, w_type, N, H, kind, mean, rstd, dy, y_type, dx, dweight, dbias, g_type, flags,
                 workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_norm_bwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_norm_bwd(x or None, int(x_type), weight or None, int(w_type), int(N), int(H), int(kind),
                                        mean or None, rstd or None, dy or None, int(y_type), dx or None,
                                        dweight or None, dbias or None, int(g_type), int(flags), workspace or None,
                                        int(workspace_bytes), stream or None)


def raw_embed_workspace_bytes(N: int, H: int, V: int) -> int:
    out = ctypes.c_size_t(0)
    check(load().lmhead_logps_embed_workspace_bytes(int(N), int(H), int(V), ctypes.byref(out)))
    return int(out.value)


def raw_embed_fwd(W, w_type, ids, N, H, V, scale, y, y_type, stream) -> int:
    """Call lmhead_logps_embed_fwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_embed_fwd(W or None, int(w_type), ids or None, int(N), int(H), int(V), float(scale),
                                         y or None, int(y_type), stream or None)


def raw_embed_bwd(ids, dy, y_type, N, H, V, scale, dW, g_type, flags, workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_embed_bwd with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_embed_bwd(ids or None, dy or None, int(y_type), int(N), int(H), int(V), float(scale),
                                         dW or None, int(g_type), int(flags), workspace or None, int(workspace_bytes),
                                         stream or None)


BEAM_MAX_BEAMS = 64
BEAM_MAX_CANDIDATES = 64


def raw_beam_workspace_bytes(N: int, H: int, V: int, beams: int, candidates: int) -> int:
    out = ctypes.c_size_t(0)
    check(load().lmhead_logps_beam_workspace_bytes(int(N), int(H), int(V), int(beams), int(candidates),
                                                   ctypes.byref(out)))
    return int(out.value)


def raw_beam_step(hidden, W, scores, ended, allowed, N, H, V, beams, candidates, temperature, top_scores, top_ids,
                  top_parents, lse, workspace, workspace_bytes, stream) -> int:
    """Call lmhead_logps_beam_step with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_beam_step(hidden or None, W or None, scores or None, ended or None, allowed or None,
                                         int(N), int(H), int(V), int(beams), int(candidates), float(temperature),
                                         top_scores or None, top_ids or None, top_parents or None, lse or None,
                                         workspace or None, int(workspace_bytes), stream or None)


def raw_beam_reorder(states, out, parents, lengths, planes, rows, beams, runs, steps, step_bytes, stream) -> int:
    """Call lmhead_logps_beam_reorder with integer addresses (0 = NULL); returns the status."""
    return load().lmhead_logps_beam_reorder(states or None, out or None, parents or None, lengths or None, int(planes),
                                            int(rows), int(beams), int(runs), int(steps), int(step_bytes),
                                            stream or None)


TRACE_KERNELS = ("fwd_stats_kernel", "fwd_merge_kernel", "bwd_step_kernel", "transpose_kernel",
                 "fill_zero_kernel", "pad_rows_kernel", "bwd_step_bf16_kernel", "distill_top_kernel",
                 "distill_prep_kernel", "distill_step_kernel", "distill_post_kernel", "few_stats_kernel",
                 "few_dz_kernel", "few_grads_kernel", "norm_fwd_kernel", "norm_bwd_kernel", "norm_reduce_kernel",
                 "embed_fwd_kernel", "embed_few_kernel", "embed_sort_kernel", "embed_rows_kernel",
                 "embed_join_kernel",
                 "beam_logits_kernel", "beam_select_kernel", "beam_score_kernel", "beam_rank_kernel",
                 "beam_reorder_kernel")


def trace_enable(on: bool) -> None:
    check(load().lmhead_logps_trace_enable(1 if on else 0))


def trace_read() -> dict:
    """{kernel name: {launches, ms, flops, bytes}} of the launches recorded
    since tracing was enabled (waits for them to finish)."""
    lib = load()
    out = {}
    for k in range(len(TRACE_KERNELS)):
        n = ctypes.c_int64(0)
        ms, fl, by = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
        check(lib.lmhead_logps_trace_read(k, ctypes.byref(n), ctypes.byref(ms), ctypes.byref(fl), ctypes.byref(by)))
        out[lib.lmhead_logps_trace_kernel_name(k).decode()] = {
            "launches": int(n.value), "ms": ms.value, "flops": fl.value, "bytes": by.value}
    return out


def version() -> str:
    return load().lmhead_logps_version().decode()
