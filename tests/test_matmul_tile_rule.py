"""Which tile a product takes (a host rule): the widths that the GPU tests of each
width rely on, and its answers at the ends of its range."""
import pytest

import sink_window_video_b200 as swv
from matmul_tiles import DENSE, GROUPED, KS


@pytest.mark.parametrize("table,E", [(DENSE, 1), (GROUPED, None)], ids=["dense", "grouped"])
def test_the_cases_of_each_width_take_it(table, E):
    assert sorted({w for w, *_ in table}) == [32, 64, 128, 192, 224]
    for w, *shape in table:
        M, N = shape[:2]
        for K in KS:
            assert swv.matmul_tile(M, N, K, E or shape[2], 148) == w, (M, N, K)
    # ragged channels, ending in the first and in the second 128 of a pair's 256
    for pair in (192, 224):
        ends = {0 < s[1] % 256 <= 128 for w, *s in table if w == pair}
        assert ends == {True, False}


def test_ends_of_the_range():
    for bad in [(0, 64, 64, 1, 148), (64, 0, 64, 1, 148), (64, 64, 0, 1, 148), (64, 64, 64, 0, 148),
                (64, 64, 64, 1, 1), (64, 64, 64, 1, -5), ((1 << 24) + 1, 64, 64, 1, 148)]:
        assert swv.matmul_tile(*bad) == 0
    for sms in (2, 148, 1 << 20):
        for big in [(1 << 24, 1, 32, 1), (1, 1 << 24, 32, 1), (1, 1, 1 << 24, 1), (1, 1, 32, 1024),
                    (1 << 24, 1 << 10, 1 << 10, 1024)]:
            assert swv.matmul_tile(*big, sms) in (32, 64, 128, 192, 224)


def test_tiles_of_few_rows_stay_on_single_ctas():
    """A pair takes longer for a step along k than a CTA does for up to 128 tokens,
    so that a long K is no reason for one."""
    for M in (1, 16, 40, 100, 128):
        for N in (512, 2048, 3696, 8192):
            for K in (512, 2048, 7808, 8192, 1 << 16):
                assert swv.matmul_tile(M, N, K) <= 128, (M, N, K)
                assert swv.matmul_tile(8 * M, N, K, 8) <= 128, (M, N, K)
