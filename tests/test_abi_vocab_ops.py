"""Refusals of the embedding's, the beam step's and the reordering's entry
points on the host: documented codes before anything touches the GPU (fake
device addresses are used only on paths that fail validation), and the
workspace sizes."""
import ctypes

import pytest

from cross_entropy_amd import _native as nat

FAKE = 0x10000
MIS = FAKE + 2


def _ef(**kw):
    a = dict(W=FAKE, w_type=0, ids=FAKE, N=4, H=100, V=300, scale=1.0, y=FAKE, y_type=0, stream=0)
    a.update(kw)
    return nat.raw_embed_fwd(**a)


def _eb(**kw):
    a = dict(ids=FAKE, dy=FAKE, y_type=0, N=4, H=100, V=300, scale=1.0, dW=FAKE, g_type=1, flags=0, workspace=FAKE,
             workspace_bytes=0, stream=0)
    a.update(kw)
    return nat.raw_embed_bwd(**a)


@pytest.mark.parametrize("call", [_ef, _eb])
def test_embed_errors(call):
    assert call(N=-1) == -2
    assert call(N=1 << 31) == -2
    for H in (0, -5, 1 << 20):
        assert call(H=H) == -2
    for V in (0, -1, 1 << 31):
        assert call(V=V) == -2
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=scale) == -5
    assert call(y_type=2) == -5
    assert call(ids=0) == -1
    assert call(ids=MIS) == -6


def test_embed_forward_errors():
    assert _ef(w_type=-1) == -5
    for k in ("W", "y"):
        assert _ef(**{k: 0}) == -1
        assert _ef(**{k: FAKE + 1}) == -6
    assert _ef(w_type=1, W=MIS) == -6
    assert _ef(y_type=1, y=MIS) == -6
    assert _ef(N=0, W=0, ids=0, y=0) == 0
    assert _ef(N=1 << 28, H=128) == -6


def test_embed_backward_errors():
    assert _eb(g_type=2) == -5
    for flags in (1, 4):
        assert _eb(flags=flags) == -5
    for k in ("dy", "dW", "workspace"):
        assert _eb(**{k: 0}) == -1
        assert _eb(**{k: FAKE + 1}) == -6
    assert _eb(workspace=FAKE + 8) == -6
    assert _eb(dW=MIS) == -6
    assert _eb(g_type=0, dW=MIS) == -4
    assert _eb(y_type=1, dy=MIS) == -6
    assert _eb(N=1 << 23) == -6
    assert _eb(V=1 << 23) == -6
    assert _eb(workspace_bytes=nat.raw_embed_workspace_bytes(4, 100, 300) - 1) == -4
    assert _eb(N=0, flags=2, ids=0, dy=0, dW=0, workspace=0) == 0
    assert _eb(N=0, ids=0, dy=0, dW=0) == -1


def test_embed_workspace():
    q = nat.raw_embed_workspace_bytes
    for bad in ((-1, 64, 10), (4, 0, 10), (4, 64, 0), (1 << 23, 64, 10), (4, 64, 1 << 23)):
        with pytest.raises(nat.LmheadError):
            q(*bad)
    assert nat.load().lmhead_logps_embed_workspace_bytes(1, 1, 1, ctypes.cast(None, ctypes.POINTER(ctypes.c_size_t))) == -1
    for N in (0, 1, 63, 64, 65, 4096, 65536, (1 << 23) - 256):
        for V in (1, 255, 256, 257, 151936, 524288, 524289, (1 << 23) - 256):
            for H in (1, 1001, 2560):
                # 20 bytes a token and a partial row per 16 of them, a byte a word, the classes' counters
                assert q(N, H, V) <= 21 * N + (N // 16 + 2) * H * 4 + V + 4096 * 13 + 2048
                assert q(N, H, V) >= (20 * N + V if N > 2048 else 16 * N)


def _bs(**kw):
    a = dict(hidden=FAKE, W=FAKE, scores=FAKE, ended=FAKE, allowed=FAKE, N=64, H=128, V=300, beams=4, candidates=8,
             temperature=1.0, top_scores=FAKE, top_ids=FAKE, top_parents=FAKE, lse=FAKE, workspace=FAKE,
             workspace_bytes=0, stream=0)
    a.update(kw)
    return nat.raw_beam_step(**a)


def test_beam_step_errors():
    assert _bs(N=-4) == -2
    assert _bs(N=1 << 31) == -2
    assert _bs(H=0) == -2
    assert _bs(V=0) == -2
    assert _bs(V=1 << 31) == -2
    assert _bs(H=96) == -6
    for beams in (0, -1, nat.BEAM_MAX_BEAMS + 1, 1 << 40):
        assert _bs(beams=beams) == -2
    assert _bs(beams=5) == -2                      # 64 rows are no groups of 5
    for C in (0, -1, nat.BEAM_MAX_CANDIDATES + 1, 1 << 40):
        assert _bs(candidates=C) == -2
    assert _bs(N=1 << 23) == -6
    assert _bs(beams=64, V=1 << 25) == -6
    assert _bs(N=1 << 20, beams=1) == -6           # groups times what each scores
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert _bs(temperature=T) == -5
    for k in ("hidden", "W", "scores", "top_scores", "top_ids", "top_parents", "lse", "workspace"):
        assert _bs(**{k: 0}) == -1, k
    for k in ("hidden", "W", "workspace"):
        assert _bs(**{k: FAKE + 8}) == -6, k
    for k in ("scores", "ended", "allowed", "top_scores", "top_ids", "top_parents", "lse"):
        assert _bs(**{k: MIS}) == -6, k
    assert _bs(ended=0, allowed=0) == -4           # optional
    need = nat.raw_beam_workspace_bytes(64, 128, 300, 4, 8)
    assert _bs(workspace_bytes=need - 1) == -4
    none = {k: 0 for k in ("hidden", "W", "scores", "ended", "allowed", "top_scores", "top_ids", "top_parents", "lse",
                           "workspace")}
    assert _bs(N=0, **none) == 0


def test_beam_workspace():
    q = nat.raw_beam_workspace_bytes
    for bad in ((64, 128, 300, 5, 8), (64, 128, 300, 4, 0), (64, 100, 300, 4, 8), (64, 128, 300, 65, 8), (-4, 128, 300, 4, 8)):
        with pytest.raises(nat.LmheadError):
            q(*bad)
    assert nat.load().lmhead_logps_beam_workspace_bytes(4, 64, 10, 1, 1, ctypes.cast(None, ctypes.POINTER(ctypes.c_size_t))) == -1
    up = lambda n, m: -(-n // m) * m  # noqa: E731
    for N in (0, 1, 4, 64, 65, 128, 129, 256, 257, 1024, 100000):
        for V in (1, 16, 17, 4096, 12289, 151936, 1 << 22):
            b = q(N, 2560, V, 1, 8)
            assert 4 * N * -(-V // 16) <= b
            # for rows rounded up to 64, or 256 above 64 of them: blocks of 16 words, sections and records of at least
            # 64, all of whole tiles of 256; and the groups' chosen blocks
            ld, v = up(max(N, 1), 64 if N <= 128 else 256), up(V, 256)
            assert b <= ld * (4 * v / 16 + 12 * (v / 64 + 256)) + N * (8 + 80 * 132 + 8) + 4096


def _br(**kw):
    a = dict(states=FAKE, out=FAKE, parents=FAKE, lengths=0, planes=2, rows=8, beams=4, runs=1, steps=10, step_bytes=2,
             stream=0)
    a.update(kw)
    return nat.raw_beam_reorder(**a)


def test_beam_reorder_errors():
    for beams in (0, -1, nat.BEAM_MAX_BEAMS + 1, 5):
        assert _br(beams=beams) == -2, beams
    for k in ("planes", "rows", "runs", "steps", "step_bytes"):
        assert _br(**{k: -4}) == -2, k
        assert _br(**{k: 0}) == 0, k               # nothing to do
    for k in ("states", "out", "parents"):
        assert _br(**{k: 0}) == -1, k
    assert _br(parents=MIS) == -6
    assert _br(lengths=MIS) == -6
    size = 2 * 8 * 10 * 2
    for off in (1, 2, size - 1):
        assert _br(out=FAKE + off) == -5
        assert _br(states=FAKE + off) == -5
    assert _br(steps=1 << 40) == -6
    assert _br(steps=1 << 62, step_bytes=1 << 62) == -6
    assert _br(rows=1 << 33, steps=1, planes=1) == -6
    assert _br(rows=1 << 30, steps=1, planes=1) == -6
    assert _br(steps=1 << 35, step_bytes=1, planes=1) == -6
    assert _br(beams=1, planes=1, rows=1 << 24, steps=1, step_bytes=1) == -6     # a workgroup each
    assert _br(beams=1, planes=1 << 10, rows=1 << 14, steps=1, step_bytes=1) == -6
