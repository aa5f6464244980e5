"""Variants of the feed-forward tile kernel that the sizes of test_gpu_ffn.py do not reach, by its own check: up to 128
tokens with so many columns that a launch has more than six rounds of tiles, and 25 to 48 tokens with a split K, whose
partial sums are counted and whose rows take two of an accumulator's lane quarters.  Products of up to 60000 terms: the
accumulation's error stays below 60000 / 16 steps of 2^-23 of the magnitudes, 4.5e-4, against 2^-8 for the operands'
rounding."""
import pytest

from test_gpu_ffn import check, mok  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I", [(5, 64, 30000), (16, 64, 30000), (100, 72, 30008), (128, 64, 29312), (16, 60000, 64),
                                   (100, 60008, 72)])
def test_more_than_six_rounds_of_tiles(mok, T, H, I):  # noqa: F811
    check(mok, T, H, I, "silu" if T % 5 else "gelu")


@pytest.mark.parametrize("T,H,I", [(25, 1024, 512), (33, 1024, 512), (40, 1024, 512), (48, 2048, 1000), (49, 1024, 512)])
def test_counted_partials_of_two_lane_quarters(mok, T, H, I):  # noqa: F811
    check(mok, T, H, I, "gelu" if T % 5 else "silu")
