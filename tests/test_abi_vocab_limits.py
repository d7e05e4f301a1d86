"""The largest launches of the lookup and the reordering, on the host: a size
whose launch would hold 2^32 threads is refused, the one below it is not (a null
pointer, which is looked at next, tells the two apart)."""
import pytest

from cross_entropy_amd import _native as nat


@pytest.mark.parametrize("N,H,status", [((1 << 24) - 1, 2048, -1),     # 2^33 - 512 groups of four elements, 512 a workgroup
                                        (599479, 4 * 14329, -6),       # 2^33 - 1
                                        (599479, 4 * 14329 - 3, -6),   # a row's last group may be cut short
                                        (1 << 24, 2048, -6)])
def test_largest_lookup(N, H, status):
    for w_type in (0, 1):
        for y_type in (0, 1):
            assert nat.raw_embed_fwd(0, w_type, 0x10000, N, H, 300, 1.0, 0x10000, y_type, 0) == status


@pytest.mark.parametrize("rows,status", [((1 << 24) - 8, -1), ((1 << 24) - 7, -6), ((1 << 24) - 1, -6), (1 << 24, -6)])
def test_largest_reordering(rows, status):
    """A workgroup a row; launches have a multiple of 8 of them."""
    assert nat.raw_beam_reorder(0, 0x10000, 0x10000, 0, 1, rows, 1, 1, 1, 1, 0) == status
