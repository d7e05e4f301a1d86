"""The workspace of the distillation's backward for few tokens, within what the
header says of it at every size of a hidden row."""
import pytest

from cross_entropy_amd import _native as nat


def _partials(N, H, V, K, chunk):
    """Bytes past the special entries and the cotangent of few tokens."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    padded = 32 if N <= 32 else -(-N // 64) * 64
    words = 2 if N <= 64 else 1
    entries = 2 * up(4 * N) + 2 * up(4 * N * (K + 1))
    return nat.raw_distill_workspace_bytes(N, H, V, K, chunk, 1) - entries - words * up(2 * V * padded)


@pytest.mark.parametrize("H", [64, 256, 2560, 16384, 65536, 131072, (1 << 20) - 64])
def test_partials_of_dh(H):
    """At most 32 MiB, or one float32 [N, H] where that is more; at least one."""
    for N in (1, 16, 32, 33, 64, 65, 128, 192, 256):
        for V in (1, 64, 1000, 12288):
            b = _partials(N, H, V, 5, 4096)
            assert 4 * N * H <= b <= max(32 << 20, 4 * N * H + 256), (N, V, b)
    for V in (24576, 151936, (1 << 23) - 256):
        for N in (1, 32, 64):
            assert 4 * N * H <= _partials(N, H, V, 5, 4096) <= max(32 << 20, 4 * N * H + 256), (N, V)
