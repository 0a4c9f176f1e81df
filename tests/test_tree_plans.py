"""Which tiles trees get, from the size of their workspace.  Host code only."""
import pytest

w4 = pytest.importorskip("w4a16_mixed_precision_offline_amd")


def test_one_tile_of_a_few_blocks_is_narrow():
    """Tiles of 128 columns are joined by a second launch, which takes two stripes for granted: what would be
    one tile in one stripe (one sequence and kv head, 128 columns, twelve blocks) never has them."""
    for D in (64, 128):
        for ratio in (1, 2, 5, 16, 128):
            for new in range(1, 128 // ratio + 1):
                for length in (1, 32, 33, 200, 384):
                    for window in (0, 1, 100, 100000):
                        for tokens in (new, 4 * new):
                            got = w4.w4a16_kv4_tree_workspace_bytes(1, tokens, new, max(new, length), ratio, 1, D, window)
                            assert got <= 4 * (512 + 1024 * 16 * (D + 2)), (D, ratio, new, length, window)
    assert w4.w4a16_kv4_tree_workspace_bytes(8, 8 * 16, 16, 8192, 64, 8, 128, 0) > 4 * (512 + 1024 * 16 * 130)
