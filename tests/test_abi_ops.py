"""Refusals of the distillation and norm entry points on the host: documented
codes before anything touches the GPU (fake device addresses are used only on
paths that fail validation), and the workspace sizes."""
import ctypes

import pytest

from cross_entropy_amd import _native as nat

FAKE = 0x10000
MIS = FAKE + 2


def _fwd(**kw):
    a = dict(hidden=FAKE, W=FAKE, targets=FAKE, ids=FAKE, teacher=FAKE, teacher_type=1, teacher_lse=FAKE, N=64, H=128,
             V=300, K=5, chunk_size=16, temperature=1.0, kl=FAKE, logp=FAKE, lse=FAKE, logp_top=FAKE, workspace=FAKE,
             workspace_bytes=0, stream=0)
    a.update(kw)
    return nat.raw_distill_fwd(**a)


def _bwd(**kw):
    a = dict(hidden=FAKE, W=FAKE, targets=FAKE, ids=FAKE, teacher=FAKE, teacher_type=1, teacher_lse=FAKE, N=64, H=128,
             V=300, K=5, chunk_size=16, temperature=1.0, logp=FAKE, lse=FAKE, logp_top=FAKE, g_kl=FAKE, g_logp=FAKE,
             dh=FAKE, dW=FAKE, grad_type=0, flags=0, workspace=FAKE, workspace_bytes=0, stream=0)
    a.update(kw)
    return nat.raw_distill_bwd(**a)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_distill_shape_and_argument_errors(call):
    assert call(N=-1) == -2
    assert call(N=1 << 31) == -2
    assert call(H=0) == -2
    assert call(V=0) == -2
    assert call(V=1 << 31) == -2
    for K in (0, -1, nat.DISTILL_MAX_K + 1, 1 << 40):
        assert call(K=K) == -2, K
        assert "K must be" in nat.load().lmhead_logps_last_error().decode()
    assert call(chunk_size=0) == -3
    assert call(H=96) == -6
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        assert call(temperature=T) == -5, T
    for bad in (-1, 2):
        assert call(teacher_type=bad) == -5
    assert call(teacher_type=1, teacher=MIS) == -6
    assert call(teacher_type=0, teacher=MIS) == -4      # bf16 teachers need 2 bytes: the workspace fails next
    assert call(teacher_type=0, teacher=FAKE + 1) == -6
    for k in ("hidden", "W", "workspace"):
        assert call(**{k: FAKE + 8}) == -6, k
    for k in ("targets", "ids", "teacher_lse", "lse", "logp", "logp_top"):
        assert call(**{k: MIS}) == -6, k
    assert call(targets=0) == -5                        # logp / g_logp without targets
    assert call(teacher_lse=0) == -4                    # optional
    assert call() == -4


def test_distill_required_pointers():
    for k in ("hidden", "W", "ids", "teacher", "kl", "lse", "logp_top", "workspace"):
        assert _fwd(**{k: 0}) == -1, k
    for k in ("hidden", "W", "ids", "teacher", "lse", "logp_top", "dh", "dW", "workspace"):
        assert _bwd(**{k: 0}) == -1, k
    assert _fwd(targets=0, logp=0) == -4
    assert _bwd(targets=0, g_logp=0) == -4
    assert _bwd(g_kl=0) == -4
    assert _bwd(logp=0) == -5
    assert _bwd(logp=0, g_logp=0) == -4
    assert _bwd(grad_type=2) == -5
    assert _bwd(flags=4) == -5
    assert _bwd(dh=FAKE + 4) == -6
    assert _bwd(dW=FAKE + 4) == -6
    assert _bwd(N=(1 << 23) - 255) == -6
    assert _bwd(V=1 << 23) == -6
    none = {k: 0 for k in ("hidden", "W", "targets", "ids", "teacher", "teacher_lse", "kl", "logp", "lse", "logp_top",
                           "workspace")}
    assert _fwd(N=0, **none) == 0


def test_distill_workspace():
    q = nat.raw_distill_workspace_bytes
    shape = (64, 128, 300, 5, 16)
    need = [q(*shape, kind) for kind in (0, 1, 2)]
    assert _fwd(workspace_bytes=need[0] - 1) == -4
    assert _bwd(workspace_bytes=need[1] - 1, grad_type=1) == -4
    assert _bwd(workspace_bytes=need[2] - 1, grad_type=0) == -4
    # the forward: 16-byte records of every token, for at most a split per 64 vocabulary rows
    assert 0 < need[0] <= 64 * 16 * -(-300 // 64)
    assert q(256, 128, 151936, 5, 16, 0) <= 256 * 256 * 16
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    # the backward: the head's, the special entries, at most 64 partials of a block's dh and 16 of its dW
    for N, H, V, chunk in ((64, 128, 300, 16), (300, 1024, 151936, 512), (256, 256, 4096, 512), (5000, 2560, 9000, 64),
                           (20000, 512, 16000, 64)):
        for kind in (1, 2):
            block = max(chunk, -(-(1 << 25) // V))   # blocks of 2^25 entries are always taken
            more = q(N, H, V, 5, chunk, kind) - nat.raw_workspace_bytes(N, H, V, block, kind)
            ct = up(min(N, 1 << 14))
            assert more <= (64 * ct + 16 * up(V)) * H * 4 + 8 * N + 48 * N + 4096
            assert more >= 0 or N <= 256   # few tokens have a smaller layout of their own
    # few tokens within a chunk: their whole cotangent (within a float32 [chunk, V]) and 50 MB of partials
    for N, H, V, chunk in ((1, 2560, 151936, 64), (33, 2560, 151936, 64), (64, 128, 9000, 64), (128, 512, 151936, 64),
                           (256, 16384, 16384, 128)):
        b = q(N, H, V, 5, chunk, 1)
        assert b <= max(4 * V * chunk, 4 * V * 64, 1 << 27) + 2 * H * 256 + (50 << 20) + 8 * N + 48 * N + 4096
    # a huge chunk_size is a chunk past N
    assert q(40, 64, 1000, 5, (1 << 63) - 1, 2) == q(40, 64, 1000, 5, 1 << 40, 2)
    # every size on the way between the kernels' limits
    for N in (0, 1, 16, 17, 32, 33, 64, 65, 128, 129, 192, 193, 256, 257, 5000):
        for V in (1, 63, 8192, 12288, 12289, 16384, 16385, 24576, 24577, 151936, (1 << 23) - 256):
            for chunk in (1, 31, 32, 64, 4096):
                sizes = [q(N, 64, V, 3, chunk, kind) for kind in (0, 1, 2)]
                assert 0 < sizes[0] <= sizes[1] <= sizes[2]
    # beyond 2^31 entries the sizes are still whole
    N, K = 1 << 22, 1024
    assert q(N, 64, 1000, K, 16, 1) > N * (K + 1) * 6
    for bad in ((64, 128, 300, 0, 16, 0), (64, 128, 300, 5, 0, 0), (64, 100, 300, 5, 16, 0), (64, 128, 1 << 23, 5, 16, 1),
                (64, 128, 300, 5, 16, 3)):
        with pytest.raises(nat.LmheadError):
            q(*bad)
    assert nat.load().lmhead_logps_distill_workspace_bytes(1, 64, 10, 1, 1, 0, None) == -1


def test_distill_no_tokens():
    """N = 0 with dW added into leaves it alone and needs nothing."""
    assert _bwd(N=0, flags=2, hidden=0, W=0, ids=0, teacher=0, workspace=0, dh=0, lse=0, logp_top=0) == 0
    assert _bwd(N=0, dW=0) == -1


def _nf(**kw):
    a = dict(x=FAKE, x_type=0, weight=FAKE, bias=FAKE, w_type=0, N=4, H=100, eps=1e-6, kind=0, y=FAKE, y_type=0,
             mean=FAKE, rstd=FAKE, stream=0)
    a.update(kw)
    return nat.raw_norm_fwd(**a)


def _nb(**kw):
    a = dict(x=FAKE, x_type=0, weight=FAKE, w_type=0, N=4, H=100, kind=0, mean=FAKE, rstd=FAKE, dy=FAKE, y_type=0,
             dx=FAKE, dweight=FAKE, dbias=FAKE, g_type=1, flags=0, workspace=FAKE, workspace_bytes=0, stream=0)
    a.update(kw)
    return nat.raw_norm_bwd(**a)


@pytest.mark.parametrize("call", [_nf, _nb])
def test_norm_errors(call):
    assert call(N=-1) == -2
    assert call(N=1 << 31) == -2
    assert call(H=0) == -2
    assert call(H=-5) == -2
    assert call(H=nat.NORM_MAX_H + 1) == -6
    for kind in (-1, 2):
        assert call(kind=kind) == -5
    for k in ("x_type", "y_type", "w_type"):
        assert call(**{k: 2}) == -5, k
    assert call(y_type=1) == -5                  # float32 y from bf16 x
    assert call(x=0) == -1
    assert call(x=FAKE + 1) == -6
    assert call(x_type=1, x=MIS) == -6
    assert call(weight=FAKE + 1) == -6
    assert call(w_type=1, weight=MIS) == -6
    assert call(rstd=MIS) == -6
    assert call(mean=MIS) == -6


def test_norm_forward_errors():
    assert _nf(y=0) == -1
    assert _nf(y=FAKE + 1) == -6
    assert _nf(bias=FAKE + 1) == -6
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _nf(eps=eps) == -5
    assert _nf(N=0, x=0, y=0, weight=0, bias=0, mean=0, rstd=0) == 0


def test_norm_backward_errors():
    for k in ("mean", "rstd", "dy", "dx", "workspace"):
        assert _nb(**{k: 0}) == -1, k
    assert _nb(kind=1, mean=0) == -4             # no mean for RMS: the workspace fails next
    assert _nb(g_type=2) == -5
    for flags in (1, 4):
        assert _nb(flags=flags) == -5
    assert _nb(dx=FAKE + 1) == -6
    assert _nb(dy=FAKE + 1) == -6
    assert _nb(dweight=MIS) == -6
    assert _nb(dbias=MIS) == -6
    assert _nb(g_type=0, dweight=MIS) == -4
    assert _nb(workspace=FAKE + 8) == -6
    need = nat.raw_norm_workspace_bytes(4, 100)
    assert need >= 2 * 100 * 4
    assert _nb(workspace_bytes=need - 1) == -4
    assert _nb(N=0, flags=2) == 0
    assert _nb(N=0, dweight=0, dbias=0) == 0
    for bad in ((-1, 100), (4, 0), (4, nat.NORM_MAX_H + 1)):
        with pytest.raises(nat.LmheadError):
            nat.raw_norm_workspace_bytes(*bad)
    assert nat.load().lmhead_logps_norm_workspace_bytes(1, 1, ctypes.cast(None, ctypes.POINTER(ctypes.c_size_t))) == -1
    for N in (1, 5, 100, 4096, 1 << 20, (1 << 31) - 1):   # bounded, whatever N
        assert nat.raw_norm_workspace_bytes(N, 2560) <= 64 << 20
