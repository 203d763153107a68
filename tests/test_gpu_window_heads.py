"""Attention over a sliding window with all heads of counts that do not divide 128 (marked gpu): row tiles begin inside a
token there, and one of them can need a key tile more than one whose rows begin with a token."""
import pytest
import torch

from tests.serving_reference import Batch
from tests.test_gpu_window import check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# In each of these some row tile has a token more than ceil(128 / heads), and a key tile more than so many tokens could need.
@pytest.mark.parametrize("heads,window,sinks,past,n", [
    (5, 40, 0, 77, 60), (5, 40, 0, 13, 200), (12, 55, 0, 11, 200), (20, 59, 0, 45, 200), (48, 63, 0, 3, 200), (72, 64, 0, 2, 200),
    (72, 128, 4, 57, 200), (80, 64, 0, 13, 200), (80, 128, 4, 61, 200), (88, 128, 4, 60, 200), (100, 64, 0, 9, 200),
    (100, 128, 4, 59, 200)])
def test_row_tiles_that_need_one_key_tile_more(heads, window, sinks, past, n):
    what = f"{heads} heads, window {window}, {sinks} first tokens, {n} new tokens behind {past}"
    check(Batch([n], [past + n], heads, 64, past, DEV), what, window, sinks)
    check(Batch([n, 1, 3], [past + n, 700, 90], heads, 16, past, DEV, pad_rows=1), what, window, sinks, dtype=torch.float32)


@pytest.mark.parametrize("heads,n,past,sinks", [(48, 2800, 2, 4), (48, 2800, 3, 0), (72, 1900, 0, 4), (72, 1900, 7, 0), (80, 1938, 2, 4),
                                                (80, 1938, 5, 0), (88, 1600, 7, 4), (88, 1600, 0, 0)])
def test_more_row_tiles_than_an_even_cut_takes(heads, n, past, sinks):
    assert heads * n > 1024 * 128
    b = Batch([n], [past + n], heads, 64, past, DEV)
    for window in (63, 128, 512, 1024):                    # (nothing lies behind the first token's window)
        check(b, f"{heads} heads, window {window}, {sinks} first tokens, behind {past}", window, sinks)


@pytest.mark.parametrize("heads", [3, 5, 12, 20, 48, 72, 80, 120, 200])
@pytest.mark.parametrize("window,sinks", [(40, 0), (63, 4), (64, 0), (128, 4)])
def test_pasts_of_every_place_in_a_block(heads, window, sinks):
    n = 70
    for past in range(0, 64, 1 if heads < 48 else 5):
        check(Batch([n], [past + n], heads, 64, past, DEV), f"{heads} heads, window {window}, {sinks} first tokens, behind {past}",
              window, sinks)
